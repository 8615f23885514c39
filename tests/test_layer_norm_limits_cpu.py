"""CPU: the sizes of the layer norm that the header says are refused are, those
next to them are not (a call that names no tensor fails with SSMP_ERR_NULL once
its sizes have passed), and sizes whose product passes 64 bits are refused."""
from __future__ import annotations

import pytest

from tests.test_decay_cpu import E_NULL, E_SHAPE, E_UNSUP, NULL, lib  # noqa: F401


@pytest.mark.parametrize("T,H,D,rows,sums", [
    (2, 65536, 1008, E_NULL, E_NULL),
    (2, 65536, 1009, E_NULL, E_SHAPE),      # H * ceil(D / 16) >= 2^22: the weights' gradients only
    (2, 65536, 16384, E_NULL, E_SHAPE),
    (2, 4095, 16384, E_NULL, E_NULL),
    (2, 4096, 16384, E_NULL, E_SHAPE),
    (2, 65537, 8, E_SHAPE, E_SHAPE),
    ((1 << 30) - 1, 1, 1024, E_NULL, E_NULL),
    (1 << 30, 1, 1024, E_SHAPE, E_SHAPE),   # 2^40 elements
    (1 << 30, 1 << 9, (1 << 31) - 1, E_SHAPE, E_SHAPE),  # 2^70
    (1 << 30, 1 << 9, 1 << 26, E_SHAPE, E_SHAPE),        # 2^65
    (2, 1, 16385, E_UNSUP, E_UNSUP),
])
def test_layer_norm_sizes(lib, T, H, D, rows, sums):  # noqa: F811
    w = 1 << 12
    assert lib.layer_norm_pack_fwd(NULL, NULL, w, w, NULL, NULL, NULL, T, H, D, 1, 0.0, 1e-5, NULL) == rows
    call = lambda dw, db: lib.layer_norm_pack_bwd(NULL, NULL, w, NULL, NULL, NULL, NULL, dw, db, NULL, 0, T, H, D, 1, 0.0,  # noqa: E731
                                                  1e-5, NULL)
    assert call(NULL, NULL) == rows and call(w, NULL) == sums and call(NULL, w) == sums
    assert (lib.layer_norm_pack_bwd_workspace_bytes(T, H, D) > 0) == (sums == E_NULL)

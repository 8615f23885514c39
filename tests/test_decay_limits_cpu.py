"""CPU: the sizes of the linear attention that the header says are refused are, and those next to them
are not (a call that names no tensor fails with SSMP_ERR_NULL once its sizes
have passed, before anything is launched)."""
from __future__ import annotations

import pytest

from tests.test_decay_cpu import E_NULL, E_SHAPE, NULL, bwd, fwd, lib  # noqa: F401


@pytest.mark.parametrize("sizes,inside", [
    # (T / 64 + nseq + 7) * Hv < 2^23
    (dict(T=64 * ((1 << 23) - 9) + 63, nseq=1, Hv=1, Dk=8, Dv=8), True),
    (dict(T=64 * ((1 << 23) - 8), nseq=1, Hv=1, Dk=8, Dv=8), False),
    (dict(T=100, nseq=(1 << 22) - 9, Hk=1, Hv=2, Dk=8, Dv=8), True),
    (dict(T=100, nseq=(1 << 22) - 8, Hk=1, Hv=2, Dk=8, Dv=8), False),
    # (T / 128 + nseq + 7) * Hv * ceil(Dv / 128) < 2^23
    (dict(T=128 * 8183, nseq=1, Hv=128, Dk=8, Dv=1024), True),
    (dict(T=128 * 8184, nseq=1, Hv=128, Dk=8, Dv=1024), False),
    (dict(T=1 << 20, nseq=1, Hv=128, Dk=128, Dv=1024), False),
    # a row: Hk * Dk, Hv * Dv, Hv * Dk * ceil(Dv / 128) <= 2^20
    (dict(T=5, nseq=1, Hk=1, Hv=8, Dk=8, Dv=1 << 17), True),
    (dict(T=5, nseq=1, Hk=1, Hv=8, Dk=8, Dv=(1 << 17) + 8), False),
    (dict(T=5, nseq=1, Hk=8192, Hv=8192, Dk=128, Dv=128), True),
    (dict(T=5, nseq=1, Hk=8193, Hv=8193, Dk=128, Dv=128), False),
    (dict(T=5, nseq=1, Hk=1, Hv=4097, Dk=128, Dv=136), False),
    # T * Hv * max(Dk, Dv) < 2^40
    (dict(T=(1 << 21) - 1152, nseq=1, Hk=1, Hv=1, Dk=8, Dv=1 << 16), True),
    (dict(T=1 << 25, nseq=1, Hk=1, Hv=1, Dk=8, Dv=1 << 15), False),
    (dict(T=5, nseq=1, Hk=1, Hv=65535, Dk=8, Dv=8), True),
    (dict(T=5, nseq=1, Hk=1, Hv=65536, Dk=8, Dv=8), False),
])
def test_attention_sizes(lib, sizes, inside):  # noqa: F811
    Hk, Hv = sizes.get("Hk", 1), sizes["Hv"]
    T, n, cols = sizes["T"], sizes["nseq"], -(-sizes["Dv"] // 128)
    stated = ((T // 64 + n + 7) * Hv < 1 << 23 and (T // 128 + n + 7) * Hv * cols < 1 << 23 and Hv <= 65535
              and max(Hk * sizes["Dk"], Hv * sizes["Dv"], Hv * sizes["Dk"] * cols) <= 1 << 20 and n <= 1 << 24
              and T * Hv * max(sizes["Dk"], sizes["Dv"]) < 1 << 40)
    assert stated == inside
    want = E_NULL if inside else E_SHAPE
    kw = {"Hk": 1, **sizes}
    assert fwd(lib, q=NULL, k=NULL, v=NULL, g=NULL, out=NULL, **kw) == want
    assert bwd(lib, dout=NULL, dq=NULL, dk=NULL, dv=NULL, **kw) == want
    names = ("T", "nseq", "Hk", "Hv", "Dk", "Dv")
    for f in (lib.decay_attn_pack_fwd_scratch_bytes, lib.decay_attn_pack_bwd_scratch_bytes):
        got = f(*(kw[x] for x in names))
        assert got > 0 if inside and T > 128 else inside or got == 0

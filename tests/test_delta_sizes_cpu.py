"""CPU: memory sized for the largest pack serves every smaller one: no size
query falls as the tokens or the sequences grow. And what the parts of split
sequences take, by the rule that splits them, lies inside the scratch."""
from __future__ import annotations

import ctypes
import random

import pytest

HEADS = [  # Hk, Hv, Dk, Dv
    (4, 4, 128, 128), (1, 1, 8, 8), (1, 2, 64, 72), (2, 4, 40, 200), (1, 3, 128, 64), (8, 16, 128, 128), (1, 32, 64, 64),
    (16, 32, 128, 128), (1, 1, 128, 2048),
]


@pytest.fixture(scope="module")
def lib():
    from selective_state_space_varlen_amd import binding
    return binding.load()


def queries(lib, heads):
    return {"saved": lambda T, n: lib.gated_delta_pack_saved_bytes(T, n, *heads),
            "fwd": lambda T, n: lib.gated_delta_pack_fwd_scratch_bytes(T, n, *heads, 1),
            "bwd": lambda T, n: lib.gated_delta_pack_bwd_scratch_bytes(T, n, *heads, 1)}


@pytest.mark.parametrize("heads", HEADS)
def test_rule_sizes_never_fall(lib, heads):
    tokens = sorted(set(range(0, 40000, 61)) | {64 * i + j for i in range(28, 36) for j in (-1, 0, 1)}
                    | {2048 * i for i in range(1, 40)} | {1 << 17, 1 << 18, 1 << 19})
    for name, f in queries(lib, heads).items():
        for n in (1, 2, 3, 4, 7, 8, 15, 16, 31, 32, 33, 100):
            sizes = [f(T, n) for T in tokens]
            assert sizes == sorted(sizes), (name, n)
        for T in (1, 63, 2047, 2048, 4096, 4160, 8192, 16384, 16385, 33000, 65536, 1 << 18):
            sizes = [f(T, n) for n in range(1, 130)]
            assert sizes == sorted(sizes), (name, T)


@pytest.mark.parametrize("heads", [(16, 16, 128), (1, 1, 64), (8, 0, 128), (1, 1, 8), (40, 8, 512), (3, 2, 72), (64, 64, 256)])
def test_norm_sizes_never_fall(lib, heads):
    sizes = [lib.qk_norm_pack_bwd_workspace_bytes(T, *heads) for T in list(range(0, 6000)) + [1 << 14, 1 << 20]]
    assert sizes == sorted(sizes)


def test_the_most_tokens_of_a_norm(lib):
    """Four tokens a workgroup of 256, and a launch takes fewer than 2^32 threads."""
    fake, odd = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)  # never dereferenced: every call is refused

    def forward(T):
        return lib.qk_norm_pack_fwd(fake, fake, None, None, None, None, fake, odd, T, 1, 0, 8, 0, 1, 0, 1e-6, 0, None)

    top = (1 << 26) - 4
    assert forward(top) == 8  # past the sizes' check: an unaligned pointer is what is wrong with it
    for T in (top + 1, top + 2, top + 3, 1 << 26):
        assert forward(T) == 2, T
        assert lib.qk_norm_pack_bwd_workspace_bytes(T, 1, 0, 8) == 0
    assert lib.qk_norm_pack_bwd_workspace_bytes(top, 1, 0, 8) > 0


def test_sizes_of_an_unsupported_type_are_refused():
    import torch
    import selective_state_space_varlen_amd as m
    for f in (m.gated_delta_pack_fwd_scratch_bytes, m.gated_delta_pack_bwd_scratch_bytes):
        assert f(100, 1, 1, 1, 64, 64, torch.bfloat16) > 0 and f(100, 1, 1, 1, 64, 64, torch.float32) > 0
        for dtype in (torch.float16, torch.float64):
            with pytest.raises(TypeError, match="unsupported dtype"):
                f(100, 1, 1, 1, 64, 64, dtype)


def round256(n):
    return -(-n // 256) * 256


def split_chunks(T, n, Hv, Dv):
    """Chunks of a part: what decides where few long sequences are split."""
    chains, chunks = n * Hv * -(-Dv // 64), T // 64 // n
    if chains > 32 or chunks < 32:
        return 0
    p = max(chunks * chains // 128, 4)
    while 2 * p * p < chunks:
        p += 1
    return p


@pytest.mark.parametrize("heads", HEADS)
def test_parts_fit_the_scratch(lib, heads):
    Hk, Hv, Dk, Dv = heads
    rng, split = random.Random(5), 0
    for _ in range(4000):
        T, n = int(2 ** rng.uniform(10, 21)), rng.choice([1, 1, 2, 3, 5, 8, 16, 32])
        p = split_chunks(T, n, Hv, Dv)
        dkp = 64 if Dk <= 64 else 128
        parts = (T // (64 * p) + n) * Hv * dkp * (-(-Dv // 64) * 64 + dkp) * 4 if p else 0
        slots = (T // 64 + n) * Hv
        rest = round256(slots * 1024) + 2 * round256(slots * 12288) + round256(n * 4)
        assert lib.gated_delta_pack_fwd_scratch_bytes(T, n, *heads, 1) >= rest + parts, (T, n)
        split += p > 0
    assert split or Hv * -(-Dv // 64) > 32


def find(cu, n, T, slot, size):
    """The chunk (or part) in a slot, by the device's search: 64 boundaries at a
    time, each clamped. None, or (first token, tokens, sequence, number)."""
    clamp = lambda x: min(max(x, 0), T)  # noqa: E731
    lo, hi = 0, n
    while True:
        step = -(-(hi - lo) // 64)
        at = [lo + lane * step for lane in range(64)]
        assert all(0 <= min(i, n) <= n for i in at)
        a = [clamp(cu[min(i, n)]) for i in at]
        k = max(sum(i < hi and x // size + i <= slot for i, x in zip(at, a)), 1)
        if step > 1:
            lo, hi = lo + (k - 1) * step, min(lo + k * step, hi)
            continue
        seq, first = lo + k - 1, a[k - 1]
        assert 0 <= seq < n
        end = a[k] if k < 64 else clamp(cu[seq + 1])
        number = slot - (first // size + seq)
        start = first + number * size
        if number < 0 or start >= end:
            return None
        return start, min(size, end - start), seq, number


def test_any_boundaries_lead_inside():
    """Chunks, parts and walks of whole sequences, for any content of cu_seqlens."""
    rng = random.Random(8)
    for _ in range(300):
        T, n, p = rng.choice([1, 63, 64, 65, 200, 4200]), rng.choice([1, 2, 3, 5, 70, 200]), rng.choice([4, 5, 9])
        kind = rng.randrange(3)
        if kind == 0:
            cu = sorted(rng.randint(0, T) for _ in range(n + 1))
        elif kind == 1:
            cu = [rng.randint(-T, 3 * T) for _ in range(n + 1)]
        else:
            cu = [rng.choice([2 ** 31 - 1, -2 ** 31, 0, T]) for _ in range(n + 1)]
        slots, parts = T // 64 + n, T // (64 * p) + n
        seen = 0
        for slot in range(slots):
            c = find(cu, n, T, slot, 64)
            if c:
                assert 0 <= c[0] and c[0] + c[1] <= T and 0 < c[1] <= 64
                seen += c[1]
        if kind == 0:
            assert seen == cu[-1] - cu[0]
        for part in range(parts):
            w = find(cu, n, T, part, 64 * p)
            if w:
                start, tokens, seq, number = w
                slot0 = (start - number * 64 * p) // 64 + seq + number * p
                assert 0 <= slot0 and slot0 + -(-tokens // 64) <= slots and start + tokens <= T
        for s in range(n):  # a chain over a whole sequence, and the join of its parts
            a = min(max(cu[s], 0), T)
            b = max(a, min(max(cu[s + 1], 0), T))
            assert a // 64 + s + -(-(b - a) // 64) <= slots
            assert a // (64 * p) + s + -(-(b - a) // (64 * p)) <= parts

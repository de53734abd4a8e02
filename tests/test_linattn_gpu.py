"""Linear attention with a decay for each head (prompts and single tokens) against the FP64
recurrence, element by element.

Tolerances, with u = 2^-8 (bf16) or 2^-24 (fp32) half a step of the type:
* o is rounded once to its type: u |o|.
* bf16: a source token of the same chunk reaches o through its masked score lam^(t-s) q.k,
  rounded to bf16 once; an earlier one through lam^.. v, rounded to bf16 once on its way into
  the state: u * o_score for both. The state enters its product with q as a bf16 pair, an error
  of at most u^2 = 2^-16 of it: part of o_mag. An element bound of u |o| + u o_score + 2^-16
  o_mag + (fp32 sums below).
* fp32 sums: dot products over K <= 128, chunk sums over at most 128 tokens and one more sum
  per chunk, the powers of lam rounded once (2^-24) and one product each: with n = K + 128 +
  128 + 8 * chunks roundings of at most 2^-23 each (the tensor cores may truncate, a whole step
  instead of half a one): n 2^-23 o_mag, and n 2^-23 s_mag for the state.
"""
import pytest
import torch

from oracle import linattn_oracle as LO

pytestmark = pytest.mark.gpu


def make(dev, lens, dtype, H, Hk, K, V, seed=0, init=True, decay="mixed", fused=False):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, k, v = r(T, H, K).to(dtype), (r(T, Hk, K) / K ** 0.5).to(dtype), r(T, Hk, V).to(dtype)
    if decay == "mixed":                       # from 1 (no decay) to forgetting at once
        ld = -torch.logspace(-4, 1.5, Hk)
        ld[0] = 0.0
    else:
        ld = torch.full((Hk,), float(decay))
    s0 = r(len(lens), Hk, V, K) if init else None
    d = {"q": q, "k": k, "v": v, "ld": ld, "s0": s0}
    d = {n: None if t is None else t.to(dev) for n, t in d.items()}
    if fused:                                  # q, k and v side by side in one projection's rows
        row = torch.full((T, H * K + Hk * (K + V) + 8), float("nan"), dtype=dtype, device=dev)
        a, b = H * K, H * K + Hk * K
        row[:, :a], row[:, a:b], row[:, b:b + Hk * V] = d["q"].flatten(1), d["k"].flatten(1), d["v"].flatten(1)
        d["q"], d["k"], d["v"] = (row[:, :a].unflatten(1, (H, K)), row[:, a:b].unflatten(1, (Hk, K)),
                                  row[:, b:b + Hk * V].unflatten(1, (Hk, V)))
    return d


def cu_of(lens, dev):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=dev)


def bounds(ref, dtype, K, tokens):
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    n = K + 256 + 8 * (tokens // 64 + 1)
    tol = u * ref["o"].abs() + n * 2.0 ** -23 * ref["o_mag"]
    if dtype == torch.bfloat16:
        tol = tol + u * ref["o_score"] + 2.0 ** -16 * ref["o_mag"]
    return tol + 1e-30, n * 2.0 ** -23 * ref["s_mag"] + 1e-30


def check(o, fin, ref, dtype, K, tokens):
    to, ts = bounds(ref, dtype, K, tokens)
    eo, es = (o.double().view_as(ref["o"]) - ref["o"]).abs(), (fin.double() - ref["final"]).abs()
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(fin).all())
    assert bool((eo <= to).all()), f"o: worst {(eo / to).max().item():.3g} of its bound"
    assert bool((es <= ts).all()), f"state: worst {(es / ts).max().item():.3g} of its bound"


HEADS = [(4, 4, 64, 64), (4, 4, 128, 128), (6, 2, 128, 64), (8, 1, 64, 128), (2, 2, 16, 16), (3, 3, 96, 80),
         (4, 2, 8, 120), (2, 1, 40, 24)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,Hk,K,V", HEADS)
def test_packed_prompts(ssd, cuda_dev, H, Hk, K, V, dtype):
    lens = [0, 1, 127, 128, 129, 0, 300, 2, 65, 0]
    d = make(cuda_dev, lens, dtype, H, Hk, K, V, seed=H * 100 + K)
    ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, d["s0"], lens)
    for seg in (0, 128):                       # the planner's segments, and as many as there can be
        ssd.set_segment_tokens(seg)
        try:
            o, fin = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=d["s0"], cu_seqlens=cu_of(lens, cuda_dev))
        finally:
            ssd.set_segment_tokens(0)
        ssd.device_status()
        check(o, fin, ref, dtype, K, 300)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,Hk,K,V", HEADS)
@pytest.mark.parametrize("lens", [[1] * 9, [64, 65, 0, 63, 7, 400], [32, 33, 0, 31, 7, 300], [2500, 1, 0, 33, 64, 130], [32] * 8 + [900]])
def test_short_sequences_among_long_ones(ssd, cuda_dev, H, Hk, K, V, dtype, lens):
    """Short sequences go token by token or, where they are few, through the chunks."""
    d = make(cuda_dev, lens, dtype, H, Hk, K, V, seed=17)
    ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, d["s0"], lens)
    state = d["s0"].clone()
    o, fin = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=state, final_state=state, cu_seqlens=cu_of(lens, cuda_dev))
    ssd.device_status()
    check(o, fin, ref, dtype, K, max(lens))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b,L", [(1, 1), (3, 63), (2, 128), (1, 385), (2, 700)])
def test_dense_prompts(ssd, cuda_dev, b, L, dtype):
    H, Hk, K, V = 6, 3, 64, 128
    lens = [L] * b
    d = make(cuda_dev, lens, dtype, H, Hk, K, V, seed=L, init=L % 2 == 1)
    ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], -0.25, d["s0"], lens)
    rs = lambda t: t.view(b, L, *t.shape[1:])  # noqa: E731
    for seg in (0, 256):
        ssd.set_segment_tokens(seg)
        try:
            o, fin = ssd.linear_attn_fwd(rs(d["q"]), rs(d["k"]), rs(d["v"]), d["ld"], scale=-0.25, init_state=d["s0"])
        finally:
            ssd.set_segment_tokens(0)
        ssd.device_status()
        check(o, fin, ref, dtype, K, L)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,Hk,K,V", [(8, 1, 128, 64), (6, 2, 64, 128), (2, 2, 128, 128)])
def test_many_chunks(ssd, cuda_dev, H, Hk, K, V, dtype):
    """Ten chunks in one segment and in several, with and without a partial one at the end."""
    lens = [1280, 1217]
    d = make(cuda_dev, lens, dtype, H, Hk, K, V, seed=H)
    ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, d["s0"], lens)
    for seg in (1 << 20, 384):
        ssd.set_segment_tokens(seg)
        try:
            o, fin = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=d["s0"], cu_seqlens=cu_of(lens, cuda_dev))
        finally:
            ssd.set_segment_tokens(0)
        ssd.device_status()
        check(o, fin, ref, dtype, K, 1280)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_long_prompt_keeps_the_precision_of_slow_decays(ssd, cuda_dev, dtype):
    """32,768 tokens of one head pair: the state remembers thousands of chunks."""
    L, H, K, V = 32768, 2, 64, 64
    d = make(cuda_dev, [L], dtype, H, H, K, V, seed=5, decay=-2e-6)
    o, fin = ssd.linear_attn_fwd(d["q"][None], d["k"][None], d["v"][None], d["ld"], init_state=d["s0"])
    ssd.device_status()
    S, M = d["s0"][0].double(), d["s0"][0].double().abs()
    lam = torch.exp(d["ld"].double()).view(H, 1, 1)
    t = torch.arange(L - 1, -1, -1, device=cuda_dev, dtype=torch.float64)
    w = torch.exp(d["ld"].double()[:, None] * t)                     # [H, L]
    k, v = d["k"].double(), d["v"].double()
    S = lam ** L * S + torch.einsum("ht,thv,thk->hvk", w, v, k)
    M = lam ** L * M + torch.einsum("ht,thv,thk->hvk", w, v.abs(), k.abs())
    err = (fin[0].double() - S).abs()
    # roundings: the same count per chunk as above, but only those of the path of one source
    # (its chunk's sum, then one per chunk it lives through, 2^-24 each and of random sign):
    # far below n 2^-23 with n = K + 256 + 512 chunks
    assert bool((err <= (K + 256 + 512) * 2.0 ** -23 * M).all()), (err / M).max().item()
    # and not the growth of a rounded lam^chunk: 512 * 2^-25 relative would be 1.5e-5
    assert (err.norm() / S.norm()).item() < 2e-6


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_slices_of_one_projection_and_rows_behind_the_last_sequence(ssd, cuda_dev, dtype):
    lens, H, Hk, K, V = [70, 200], 4, 2, 64, 64
    d = make(cuda_dev, lens, dtype, H, Hk, K, V, seed=3, fused=True)
    assert not d["q"].is_contiguous()
    ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, d["s0"], lens)
    o, fin = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=d["s0"], cu_seqlens=cu_of(lens, cuda_dev))
    check(o, fin, ref, dtype, K, 200)
    # a dense batch out of the same rows
    r = lambda t: t[:200].unflatten(0, (2, 100))  # noqa: E731
    o2, f2 = ssd.linear_attn_fwd(r(d["q"]), r(d["k"]), r(d["v"]), d["ld"], init_state=d["s0"])
    ssd.device_status()
    ref2 = LO.linattn(d["q"][:200], d["k"][:200], d["v"][:200], d["ld"], K ** -0.5, d["s0"], [100, 100])
    check(o2, f2, ref2, dtype, K, 100)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_other_sequences_never_see_a_non_finite_value(ssd, cuda_dev, bad):
    """NaN and infinities in one packed sequence, next to others inside the same 128-token tile."""
    lens, H, K, V = [50, 30, 200], 2, 64, 64
    d = make(cuda_dev, lens, torch.bfloat16, H, H, K, V, seed=4)
    clean = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, d["s0"], lens)
    for name in ("q", "k", "v"):
        d[name] = d[name].clone()
        d[name][50:80] = bad
    o, fin = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=d["s0"], cu_seqlens=cu_of(lens, cuda_dev))
    ssd.device_status()
    keep = torch.cat([torch.arange(50), torch.arange(80, 280)]).to(cuda_dev)
    ref = {n: t[keep] if n.startswith("o") else t[[0, 2]] for n, t in clean.items()}
    check(o[keep], fin[[0, 2]], ref, torch.bfloat16, K, 200)


def test_non_finite_values_reach_no_earlier_chunk(ssd, cuda_dev):
    L, H, K, V = 400, 2, 64, 64
    d = make(cuda_dev, [L], torch.bfloat16, H, H, K, V, seed=6)
    clean = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, d["s0"])
    d["v"] = d["v"].clone()
    d["v"][300, 0] = float("inf")              # head 0; chunk of 128 tokens from 256 on
    o, _ = ssd.linear_attn_fwd(d["q"][None], d["k"][None], d["v"][None], d["ld"], init_state=d["s0"])
    to, _ = bounds(clean, torch.bfloat16, K, L)
    ok = (o[0].double() - clean["o"]).abs() <= to
    assert bool(ok[:256].all()) and bool(ok[:, 1].all())


def test_zero_init_none_and_final_not_wanted(ssd, cuda_dev):
    lens, H, K, V = [5, 140], 2, 128, 64
    d = make(cuda_dev, lens, torch.bfloat16, H, H, K, V, seed=8, init=False)
    ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, None, lens)
    o, fin = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], cu_seqlens=cu_of(lens, cuda_dev))
    check(o, fin, ref, torch.bfloat16, K, 140)
    import ctypes
    o2 = torch.zeros_like(o)
    dims = ssd.linear_attn_dims((145,), H, H, K, V, ssd.SSD_DTYPE_BF16, 2)
    rc = ssd._lib.ssd_linear_attn_fwd(d["q"].data_ptr(), d["k"].data_ptr(), d["v"].data_ptr(), d["ld"].data_ptr(), K ** -0.5,
                                      None, None, cu_of(lens, cuda_dev).data_ptr(), o2.data_ptr(), None, None,
                                      ctypes.byref(dims), torch.cuda.current_stream().cuda_stream)
    ssd.device_status()
    assert rc == ssd.SSD_OK and torch.equal(o, o2)


@pytest.mark.parametrize("seg", [0, 128])
def test_states_in_pages_and_in_place(ssd, cuda_dev, seg):
    lens, H, K, V = [260, 0, 90, 400], 2, 64, 64
    d = make(cuda_dev, lens, torch.bfloat16, H, H, K, V, seed=9)
    ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, d["s0"], lens)
    pages = torch.tensor([6, 1, 4, 0], dtype=torch.int32, device=cuda_dev)
    pool = torch.full((8, H, V, K), 7.0, device=cuda_dev)
    pool[pages.long()] = d["s0"]
    cu = cu_of(lens, cuda_dev)
    ssd.set_segment_tokens(seg)
    try:
        o, got = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=pool, init_pages=pages, cu_seqlens=cu,
                                     final_state=pool, final_pages=pages)
        assert got is pool
        check(o, pool[pages.long()], ref, torch.bfloat16, K, 400)
        assert bool((pool[[2, 3, 5, 7]] == 7.0).all())
        # dense states replaced in place
        s = d["s0"].clone()
        o2, _ = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=s, cu_seqlens=cu, final_state=s)
        check(o2, s, ref, torch.bfloat16, K, 400)
        # -1: a zero start, a final state that is not written
        ssd.device_status()
        ip = torch.tensor([-1, 1, -1, 0], dtype=torch.int32, device=cuda_dev)
        fp = torch.tensor([-1, 2, 3, -1], dtype=torch.int32, device=cuda_dev)
        pool = torch.full((8, H, V, K), 7.0, device=cuda_dev)
        pool[1], pool[0] = d["s0"][1], d["s0"][3]
        z = d["s0"].clone()
        z[[0, 2]] = 0
        ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, z, lens)
        o, _ = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=pool, init_pages=ip, cu_seqlens=cu,
                                   final_state=pool, final_pages=fp)
        ssd.device_status()
        check(o, torch.stack([ref["final"][0].float(), pool[2], pool[3], ref["final"][3].float()]), ref, torch.bfloat16, K, 400)
        assert bool((pool[[4, 5, 6, 7]] == 7.0).all()) and torch.equal(pool[0], d["s0"][3])
    finally:
        ssd.set_segment_tokens(0)


@pytest.mark.parametrize("seg", [0, 128])
@pytest.mark.parametrize("ip,fp,kept", [
    ([0, 1, 2], [3, 3, 4], 1),                 # two sequences end in one page: the first one writes it
    ([0, 1, 2], [3, 0, 4], 1),                 # a sequence ends where another one starts
    ([0, 1, 2], [3, 9, 4], 1),                 # outside the pool
])
def test_clashing_pages_are_refused(ssd, cuda_dev, ip, fp, kept, seg):
    lens, H, K, V = [140, 20, 300], 2, 64, 64
    d = make(cuda_dev, lens, torch.bfloat16, H, H, K, V, seed=10)
    ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, d["s0"], lens)
    pool = torch.full((6, H, V, K), 7.0, device=cuda_dev)
    pool[:3] = d["s0"]
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_dev)  # noqa: E731
    ssd.device_status()
    ssd.set_segment_tokens(seg)
    try:
        o, _ = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=pool, init_pages=t(ip),
                                   cu_seqlens=cu_of(lens, cuda_dev), final_state=pool, final_pages=t(fp))
    finally:
        ssd.set_segment_tokens(0)
    with pytest.raises(ssd.SSDError, match="INVALID_ARG"):
        ssd.device_status()
    # every output and every other state is right; the refused one is not written anywhere
    check(o, torch.stack([pool[3], ref["final"][1].float(), pool[4]]), ref, torch.bfloat16, K, 300)
    assert torch.equal(pool[:3], d["s0"]) and bool((pool[5] == 7.0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_states_that_change_places_in_one_array_are_refused(ssd, cuda_dev, dtype):
    """Sequence 0 would start from state 1 and end in state 0, sequence 1 the other way round."""
    lens, H, K, V = [40, 60, 20], 2, 64, 64
    d = make(cuda_dev, lens, dtype, H, H, K, V, seed=15)
    swap = torch.tensor([1, 0, 2], dtype=torch.int32, device=cuda_dev)
    ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, d["s0"][swap.long()], lens)
    s = d["s0"].clone()
    ssd.device_status()
    o, _ = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=s, init_pages=swap, cu_seqlens=cu_of(lens, cuda_dev),
                               final_state=s)
    with pytest.raises(ssd.SSDError, match="INVALID_ARG"):
        ssd.device_status()
    assert torch.equal(s[:2], d["s0"][:2])
    check(o, torch.cat([ref["final"][:2].float(), s[2:]]), ref, dtype, K, 60)


def test_device_errors(ssd, cuda_dev):
    lens, H, K, V = [40, 24], 2, 64, 64
    d = make(cuda_dev, lens, torch.float32, H, H, K, V)
    ssd.device_status()
    o = torch.full((64, H, V), 3.0, device=cuda_dev)
    for cu in ([0, 50, 40], [1, 40, 64], [0, 40, 63]):
        ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=cuda_dev), o=o)
        with pytest.raises(ssd.SSDError, match="INVALID_ARG"):
            ssd.device_status()
        assert bool((o == 3.0).all())
    for ld in (0.5, float("nan"), float("-inf")):
        bad = d["ld"].clone()
        bad[1] = ld
        ssd.linear_attn_fwd(d["q"], d["k"], d["v"], bad, cu_seqlens=cu_of(lens, cuda_dev))
        with pytest.raises(ssd.SSDError, match="INVALID_ARG"):
            ssd.device_status()
        ssd.linear_attn_update(d["s0"], d["q"][:2], d["k"][:2], d["v"][:2], bad)
        with pytest.raises(ssd.SSDError, match="INVALID_ARG"):
            ssd.device_status()


def test_empty_calls(ssd, cuda_dev):
    ld = torch.zeros(2, device=cuda_dev)
    z = lambda *s: torch.zeros(*s, device=cuda_dev)  # noqa: E731
    s0 = torch.randn(3, 2, 32, 16, device=cuda_dev)
    o, fin = ssd.linear_attn_fwd(z(0, 2, 16), z(0, 2, 16), z(0, 2, 32), ld, init_state=s0, cu_seqlens=torch.zeros(4, dtype=torch.int32, device=cuda_dev))
    assert o.shape == (0, 2, 32) and torch.equal(fin, s0)
    o, fin = ssd.linear_attn_fwd(z(3, 0, 2, 16), z(3, 0, 2, 16), z(3, 0, 2, 32), ld, init_state=s0)
    assert torch.equal(fin, s0)
    o, fin = ssd.linear_attn_fwd(z(0, 5, 2, 16), z(0, 5, 2, 16), z(0, 5, 2, 32), ld)
    assert fin.shape == (0, 2, 32, 16)
    assert ssd.linear_attn_update(z(0, 2, 32, 16), z(0, 2, 16), z(0, 2, 16), z(0, 2, 32), ld).shape == (0, 2, 32)
    ssd.device_status()


def test_caller_workspace(ssd, cuda_dev):
    lens, H, K, V = [300, 500], 2, 64, 64
    d = make(cuda_dev, lens, torch.bfloat16, H, H, K, V)
    ssd.set_segment_tokens(128)
    try:
        o, f = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], cu_seqlens=cu_of(lens, cuda_dev))
        n = ssd.linear_attn_workspace_size(ssd.linear_attn_dims((800,), H, H, K, V, ssd.SSD_DTYPE_BF16, 2))
        ws = torch.empty(n, dtype=torch.uint8, device=cuda_dev)
        o2, f2 = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], cu_seqlens=cu_of(lens, cuda_dev), workspace=ws)
        with pytest.raises(ssd.SSDError, match="INVALID_ARG"):
            ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], cu_seqlens=cu_of(lens, cuda_dev), workspace=ws[:n // 2])
    finally:
        ssd.set_segment_tokens(0)
    ssd.device_status()
    assert torch.equal(o, o2) and torch.equal(f, f2)


# --------------------------------------------------------------------------------- single tokens
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,Hk,K,V", HEADS)
@pytest.mark.parametrize("b", [1, 5])
def test_single_tokens(ssd, cuda_dev, H, Hk, K, V, dtype, b):
    """Three steps in a row against the recurrence: u |o| for the result and (K + 8) 2^-24 of
    the magnitudes a step for the fp32 sums."""
    n = 3
    d = make(cuda_dev, [n] * b, dtype, H, Hk, K, V, seed=K + V)
    ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, d["s0"], [n] * b)
    s = d["s0"].clone()
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    for t in range(n):
        i = torch.arange(b, device=cuda_dev) * n + t
        o = ssd.linear_attn_update(s, d["q"][i], d["k"][i], d["v"][i], d["ld"])
        tol = u * ref["o"][i].abs() + n * (K + 8) * 2.0 ** -24 * ref["o_mag"][i] + 1e-30
        assert bool(((o.double() - ref["o"][i]).abs() <= tol).all())
    ssd.device_status()
    assert bool(((s.double() - ref["final"]).abs() <= n * 8 * 2.0 ** -24 * ref["s_mag"] + 1e-30).all())


def test_padded_batch_strided_rows_and_pages(ssd, cuda_dev):
    H, Hk, K, V, b = 8, 2, 128, 96, 6
    d = make(cuda_dev, [1] * b, torch.bfloat16, H, Hk, K, V, seed=2, fused=True)
    pages = torch.tensor([3, -1, 0, 7, -1, 5], dtype=torch.int32, device=cuda_dev)
    on = pages >= 0
    pool = torch.randn(9, Hk, V, K, device=cuda_dev)
    before = pool.clone()
    s0 = pool[pages.clamp(min=0).long()].clone()
    ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, s0, [1] * b)
    o = torch.full((b, H, V), 5.0, dtype=torch.bfloat16, device=cuda_dev)
    ssd.linear_attn_update(pool, d["q"], d["k"], d["v"], d["ld"], pages=pages, o=o)
    ssd.device_status()
    tol = 2.0 ** -8 * ref["o"].abs() + (K + 8) * 2.0 ** -24 * ref["o_mag"]
    assert bool(((o.double() - ref["o"]).abs() <= tol)[on].all())
    assert bool((o[~on] == 5.0).all())                                   # padded rows are left as they were
    got = pool[pages[on].long()].double()
    assert bool(((got - ref["final"][on]).abs() <= 8 * 2.0 ** -24 * ref["s_mag"][on]).all())
    others = [1, 2, 4, 6, 8]
    assert torch.equal(pool[others], before[others])


def test_a_page_named_twice_and_pages_out_of_range(ssd, cuda_dev):
    H, K, V, b = 2, 64, 64, 4
    d = make(cuda_dev, [1] * b, torch.float32, H, H, K, V, seed=1)
    pool = torch.randn(4, H, V, K, device=cuda_dev)
    before = pool.clone()
    one = pool.clone()
    want = ssd.linear_attn_update(one, d["q"][:1], d["k"][:1], d["v"][:1], d["ld"], pages=torch.tensor([2], dtype=torch.int32, device=cuda_dev))
    ssd.device_status()
    o = torch.full((b, H, V), 5.0, device=cuda_dev)
    ssd.linear_attn_update(pool, d["q"], d["k"], d["v"], d["ld"], pages=torch.tensor([2, 2, 4, -7], dtype=torch.int32, device=cuda_dev), o=o)
    with pytest.raises(ssd.SSDError, match="INVALID_ARG"):
        ssd.device_status()
    assert torch.equal(o[0], want[0]) and bool((o[1:] == 5.0).all())
    assert torch.equal(pool, one) and torch.equal(pool[[0, 1, 3]], before[[0, 1, 3]])


@pytest.mark.parametrize("shift", [0, 1, 3])
def test_large_batches_of_small_states(ssd, cuda_dev, shift):
    """Several rows in one block; a page named again far down the list, which may start anywhere."""
    b, H, K, V = 1030, 3, 16, 24
    d = make(cuda_dev, [1] * b, torch.float32, H, H, K, V, seed=21)
    ids = torch.randperm(b + 10, device=cuda_dev)[:b].int()
    pool = torch.zeros(b + 10, H, V, K, device=cuda_dev)
    pool[ids.long()] = d["s0"]
    hold = torch.empty(b + shift, dtype=torch.int32, device=cuda_dev)
    pages = hold[shift:]
    pages.copy_(ids)
    ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, d["s0"], [1] * b)
    twice = [(1029, 0), (1000, 640)]                 # these rows name the pages of those
    for late, early in twice:
        pages[late] = pages[early]
    before = pool.clone()
    o = ssd.linear_attn_update(pool, d["q"], d["k"], d["v"], d["ld"], pages=pages, o=torch.full((b, H, V), 5.0, device=cuda_dev))
    with pytest.raises(ssd.SSDError, match="INVALID_ARG"):
        ssd.device_status()
    ok = torch.ones(b, dtype=torch.bool, device=cuda_dev)
    for late, _ in twice:
        ok[late] = False
        assert bool((o[late] == 5.0).all()) and torch.equal(pool[ids[late]], before[ids[late]])
    check(o[ok], pool[ids.long()][ok], {n: t[ok] for n, t in ref.items()}, torch.float32, K, 1)


def test_offsets_past_32_bits(ssd, cuda_dev):
    """A pool of 2^31 state elements and more: single tokens and prompts on its last pages."""
    H, K, V, n = 64, 128, 128, 2100                  # 4 MiB a page, 8.8 GB
    lens = [1, 130]
    d = make(cuda_dev, lens, torch.bfloat16, H, H, K, V, seed=16, decay=-0.1)
    pool = torch.empty(n, H, V, K, device=cuda_dev)
    assert pool.numel() > 1 << 31
    pages = torch.tensor([n - 1, n - 2], dtype=torch.int32, device=cuda_dev)
    pool[pages.long()] = d["s0"]
    one = [d[x][:2].contiguous() for x in "qkv"]
    ref = LO.linattn(*one, d["ld"], K ** -0.5, d["s0"], [1, 1])
    o = ssd.linear_attn_update(pool, *one, d["ld"], pages=pages)
    ssd.device_status()
    tol = 2.0 ** -8 * ref["o"].abs() + (K + 8) * 2.0 ** -24 * ref["o_mag"]
    assert bool(((o.double() - ref["o"]).abs() <= tol).all())
    assert bool(((pool[pages.long()].double() - ref["final"]).abs() <= 8 * 2.0 ** -24 * ref["s_mag"]).all())
    pool[pages.long()] = d["s0"]
    ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, d["s0"], lens)
    o, _ = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=pool, init_pages=pages, cu_seqlens=cu_of(lens, cuda_dev),
                               final_state=pool, final_pages=pages)
    ssd.device_status()
    check(o, pool[pages.long()], ref, torch.bfloat16, K, 130)


# --------------------------------------------------------------------------------- together
def test_prompt_then_tokens_equals_one_prompt(ssd, cuda_dev):
    lens, more, H, Hk, K, V = [130, 7, 256], 4, 4, 2, 64, 64
    full = [n + more for n in lens]
    d = make(cuda_dev, full, torch.bfloat16, H, Hk, K, V, seed=12)
    ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, None, full)
    start = [sum(full[:i]) for i in range(3)]
    head = torch.cat([torch.arange(s, s + n) for s, n in zip(start, lens)]).to(cuda_dev)
    pages = torch.tensor([2, 0, 3], dtype=torch.int32, device=cuda_dev)
    pool = torch.zeros(4, Hk, V, K, device=cuda_dev)
    o, _ = ssd.linear_attn_fwd(d["q"][head], d["k"][head], d["v"][head], d["ld"], cu_seqlens=cu_of(lens, cuda_dev),
                               final_state=pool, final_pages=pages)
    got = torch.empty_like(ref["o"])
    got[head] = o.double()
    for t in range(more):
        row = torch.tensor([s + n + t for s, n in zip(start, lens)], device=cuda_dev)
        got[row] = ssd.linear_attn_update(pool, d["q"][row], d["k"][row], d["v"][row], d["ld"], pages=pages).double()
    ssd.device_status()
    check(got, pool[pages.long()], ref, torch.bfloat16, K, 300)


def test_other_streams_and_two_calls_at_once(ssd, cuda_dev):
    lens, H, K, V = [900, 300], 4, 64, 64
    ds = [make(cuda_dev, lens, torch.bfloat16, H, H, K, V, seed=s) for s in (21, 22)]
    cu = cu_of(lens, cuda_dev)
    ssd.set_segment_tokens(256)
    try:
        want = [ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=d["s0"], cu_seqlens=cu) for d in ds]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in ds]
        got = [[] for _ in ds]
        for _ in range(5):
            for i, (d, st) in enumerate(zip(ds, streams)):
                with torch.cuda.stream(st):
                    got[i].append(ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=d["s0"], cu_seqlens=cu))
        torch.cuda.synchronize()
    finally:
        ssd.set_segment_tokens(0)
    ssd.device_status()
    for w, g in zip(want, got):
        for o, f in g:
            assert torch.equal(o, w[0]) and torch.equal(f, w[1])


def test_captured_and_replayed(ssd, cuda_dev):
    lens, H, K, V = [400, 90], 2, 64, 64
    d = make(cuda_dev, lens, torch.bfloat16, H, H, K, V, seed=31)
    cu = cu_of(lens, cuda_dev)
    pages = torch.tensor([1, 0], dtype=torch.int32, device=cuda_dev)
    pool = torch.zeros(2, H, V, K, device=cuda_dev)
    last = torch.tensor([399, 489], device=cuda_dev)
    one = [d[n][last].contiguous() for n in "qkv"]
    o2 = torch.empty(2, H, V, dtype=torch.bfloat16, device=cuda_dev)

    def step():
        o, _ = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], cu_seqlens=cu, final_state=pool, final_pages=pages)
        ssd.linear_attn_update(pool, *one, d["ld"], pages=pages, o=o2)
        return o

    ssd.set_segment_tokens(128)
    try:
        want, want2, wpool = step().clone(), o2.clone(), pool.clone()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = step()
    finally:
        ssd.set_segment_tokens(0)
    for seed in (31, 32):                      # new inputs through the same addresses
        new = make(cuda_dev, lens, torch.bfloat16, H, H, K, V, seed=seed)
        for n in "qkv":
            d[n].copy_(new[n])
        for a, n in zip(one, "qkv"):
            a.copy_(new[n][last])
        g.replay()
        torch.cuda.synchronize()
        if seed == 31:
            assert torch.equal(o, want) and torch.equal(o2, want2) and torch.equal(pool, wpool)
        else:
            ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, None, lens)
            to, _ = bounds(ref, torch.bfloat16, K, 400)
            assert bool(((o.double() - ref["o"]).abs() <= to).all())
    ssd.device_status()


def test_two_captured_prompts_replay_at_once(ssd, cuda_dev):
    """Two graphs, each with a scratch of its own, replayed side by side on two streams."""
    lens, H, K, V = [900, 30, 700], 4, 64, 64
    cu, calls = cu_of(lens, cuda_dev), []
    for seed in (31, 32):
        d = make(cuda_dev, lens, torch.bfloat16, H, H, K, V, seed=seed)
        ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, d["s0"], lens)
        run = lambda d=d: ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=d["s0"], cu_seqlens=cu)  # noqa: E731
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        calls.append((torch.cuda.Stream(), graph, out, ref, d))       # the graph reads d again
    for _ in range(3):
        for st, graph, *_ in calls:
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    ssd.device_status()
    for _st, _graph, (o, fin), ref, _d in calls:
        check(o, fin, ref, torch.bfloat16, K, 900)


def test_refusals_of_the_binding(ssd, cuda_dev):
    d = make(cuda_dev, [32], torch.bfloat16, 4, 2, 64, 64)
    cu = cu_of([32], cuda_dev)
    call = lambda **kw: ssd.linear_attn_fwd(**{**dict(q=d["q"], k=d["k"], v=d["v"], log_decay=d["ld"], cu_seqlens=cu), **kw})  # noqa: E731
    for kw, err in [(dict(q=d["q"].float()), TypeError), (dict(k=d["k"][:31]), ValueError), (dict(cu_seqlens=None), ValueError),
                    (dict(log_decay=d["ld"].double()), TypeError), (dict(log_decay=d["ld"][:1]), ValueError),
                    (dict(q=d["q"].transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                    (dict(init_pages=cu[:1]), ValueError), (dict(final_pages=cu[:1]), ValueError),
                    (dict(init_state=d["s0"].double()), TypeError), (dict(q=d["q"].half()), TypeError),
                    (dict(q=d["q"].cpu()), ValueError), (dict(cu_seqlens=cu.long()), TypeError),
                    (dict(o=torch.empty(32, 4, 32, dtype=torch.bfloat16, device=cuda_dev)), ValueError)]:
        with pytest.raises(err):
            call(**kw)
    with pytest.raises(ValueError, match="workspace"):
        call(workspace=torch.empty(1 << 20, dtype=torch.uint8))
    off = torch.empty(32 * 4 * 64 + 1, dtype=torch.bfloat16, device=cuda_dev)[1:].view(32, 4, 64)
    with pytest.raises(ssd.SSDError, match="INVALID_ARG"):
        call(q=off)
    with pytest.raises(ssd.SSDError, match="UNSUPPORTED"):       # rows of 4 * 64 + 4 elements: not 16-byte steps
        call(q=torch.empty(32, 260, dtype=torch.bfloat16, device=cuda_dev)[:, :256].unflatten(1, (4, 64)))
    for K, V in ((72, 136), (12, 16), (136, 64)):
        z = lambda n: torch.zeros(4, 2, n, device=cuda_dev)  # noqa: E731
        with pytest.raises(ssd.SSDError, match="UNSUPPORTED"):
            ssd.linear_attn_fwd(z(K), z(K), z(V), d["ld"], cu_seqlens=cu_of([4], cuda_dev))
    ssd.device_status()


@pytest.mark.parametrize("stalled_pass", [1, 2])
def test_wait_runs_out_and_context_stays_usable(ssd, cuda_dev, stalled_pass):
    """The test hook makes one pass's UMMA warp wait for a barrier that nothing arrives at: the
    bounded waits end the call, SSD_ERR_TIMEOUT is latched and the next call is right."""
    lens, H, K, V = [300, 40], 2, 64, 64
    d = make(cuda_dev, lens, torch.bfloat16, H, H, K, V, seed=14)
    cu = cu_of(lens, cuda_dev)
    ssd.device_status()
    ssd.test_stall(stalled_pass)
    try:
        ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=d["s0"], cu_seqlens=cu)
        torch.cuda.synchronize()
        with pytest.raises(ssd.SSDError, match="TIMEOUT"):
            ssd.device_status()
    finally:
        ssd.test_stall(0)
    ssd.device_status()
    o, fin = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=d["s0"], cu_seqlens=cu)
    ssd.device_status()
    ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, d["s0"], lens)
    check(o, fin, ref, torch.bfloat16, K, 300)


def test_expanded_inputs_are_refused(ssd, cuda_dev):
    """Tokens that share memory: refused by the binding before any launch."""
    H, Hk, K, V = 4, 2, 64, 64
    d = make(cuda_dev, [12], torch.bfloat16, H, Hk, K, V)
    one = {n: d[n][:1] for n in "qkv"}
    cu = cu_of([12], cuda_dev)
    state = torch.zeros(12, Hk, V, K, device=cuda_dev)
    for n in "qkv":
        wide = one[n].expand(12, *one[n].shape[1:])
        packed = {**{m: d[m] for m in "qkv"}, n: wide}
        with pytest.raises(ValueError, match="share memory"):
            ssd.linear_attn_fwd(**packed, log_decay=d["ld"], cu_seqlens=cu)
        for b, L in ((1, 12), (3, 4), (12, 1)):
            with pytest.raises(ValueError, match="share memory"):
                ssd.linear_attn_fwd(**{m: t.unflatten(0, (b, L)) if m != n else one[n].expand(b, L, *t.shape[1:])
                                       for m, t in packed.items()}, log_decay=d["ld"])
        with pytest.raises(ValueError, match="share memory"):
            ssd.linear_attn_update(state, **packed, log_decay=d["ld"])
    ssd.device_status()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R", [1, 2])
def test_the_decay_itself(ssd, cuda_dev, dtype, R):
    """Keys of zero, so that a state is only decayed: final = lam^n S_0, for decays from none to
    past the smallest float, one token at a time, in short prompts and in chunks.
    Tolerance per token: exp and expm1 within one unit of their last place (2^-23 of lam; expm1 at
    lam >= 1/2 half of that), the rest of the step three roundings of 2^-24, of which two only
    touch the low part: below 2^-22. Where lam S_0 is subnormal: 2^-149 for a unit of lam and half
    of it for each rounding, 2^-148 (1 + |S_0|) in all."""
    decays = [0.0, -1e-6, -0.01, -0.5, -0.693, -0.6932, -0.7, -1.0, -3.0, -8.0, -12.0, -17.0, -20.0, -40.0, -80.0, -86.0, -95.0, -110.0]
    Hk, K, V = len(decays), 24, 40
    ld = torch.tensor(decays, device=cuda_dev)
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).to(cuda_dev)  # noqa: E731
    for lens in ([1], [3, 1], [1, 600, 2]):                # the last through the chunks
        T = sum(lens)
        q, k, v = r(T, Hk * R, K), torch.zeros(T, Hk, K, dtype=dtype, device=cuda_dev), r(T, Hk, V)
        s0 = r(len(lens), Hk, V, K).float()
        _, fin = ssd.linear_attn_fwd(q, k, v, ld, init_state=s0, cu_seqlens=cu_of(lens, cuda_dev))
        got = [(fin, lens)]
        if lens == [1]:
            state = s0.clone()
            ssd.linear_attn_update(state, q, k, v, ld)
            got.append((state, lens))
        ssd.device_status()
        for x, ns in got:
            n = torch.tensor(ns, device=cuda_dev, dtype=torch.float64).view(-1, 1, 1, 1)
            ref = s0.double() * torch.exp(n * ld.double().view(1, -1, 1, 1))
            bad = (x.double() - ref).abs() > n * (2.0 ** -22 * ref.abs() + 2.0 ** -148 * (1 + s0.double().abs()))
            assert not bool(bad.any()), (lens, [decays[i] for i in bad.any(3).any(2).any(0).nonzero().flatten().tolist()])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [20, 900])                   # token by token, and in chunks
def test_states_of_empty_sequences_are_copied(ssd, cuda_dev, dtype, n):
    lens, Hk, K, V = [0, n, 0, 0], 2, 64, 72
    d = make(cuda_dev, lens, dtype, Hk, Hk, K, V, seed=4)
    for i, x in enumerate((float("inf"), -float("inf"), float("nan"), -0.0, 1e-45, 3.4e38)):
        d["s0"][0, :, 7 * i, 5 * i] = x
        d["s0"][3, :, V - 1 - i, K - 1] = x
    pages = torch.tensor([3, 1, -1, 0], dtype=torch.int32, device=cuda_dev)
    for init, ip, want in ((d["s0"], None, d["s0"]), (d["s0"], pages, d["s0"][[3, 1, 2, 0]])):
        _, fin = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=init, init_pages=ip, cu_seqlens=cu_of(lens, cuda_dev))
        ssd.device_status()
        for s in (0, 3):
            assert torch.equal(fin[s].view(torch.int32), want[s].view(torch.int32))
        assert ip is None or not bool(fin[2].any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_non_finite_state_stays_in_its_row(ssd, cuda_dev, dtype, bad):
    """It makes its own element of the final state and its row of V in its head's outputs
    non-finite; everything else is bit for bit what it is without it."""
    H, Hk, K, V, hk, row, col = 4, 2, 64, 72, 1, 65, 9
    hit = slice(hk * H // Hk, (hk + 1) * H // Hk)
    for lens in ([1, 1], [5, 30], [700, 300]):             # tokens, token by token, chunks of several segments
        d = make(cuda_dev, lens, dtype, H, Hk, K, V, seed=6, decay=-0.01)
        for single in ([False, True] if lens == [1, 1] else [False]):
            out = []
            for x in (None, bad):
                s0 = d["s0"].clone()
                if x is not None:
                    s0[1, hk, row, col] = x
                if single:
                    out.append((ssd.linear_attn_update(s0, d["q"], d["k"], d["v"], d["ld"]), s0))
                else:
                    ssd.set_segment_tokens(256)
                    try:
                        out.append(ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=s0, cu_seqlens=cu_of(lens, cuda_dev)))
                    finally:
                        ssd.set_segment_tokens(0)
            ssd.device_status()
            (o, f), (o2, f2) = out
            assert not bool(torch.isfinite(o2[lens[0]:, hit, row]).any()) and not bool(torch.isfinite(f2[1, hk, row, col]))
            o2[lens[0]:, hit, row], f2[1, hk, row, col] = o[lens[0]:, hit, row], f[1, hk, row, col]
            assert torch.equal(o, o2) and torch.equal(f, f2)


def at_once(jobs, times):
    """Every job (a function of the library and its arguments) `times` times in a host thread of
    its own; how many of them returned an error."""
    import threading
    failed, start = [0] * len(jobs), threading.Barrier(len(jobs))

    def loop(i):
        fn, args = jobs[i]
        start.wait()
        failed[i] = sum(fn(*args) != 0 for _ in range(times))

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return failed


def test_threads_with_other_sizes(ssd, cuda_dev):
    """Calls of host threads whose kernels take different amounts of shared memory."""
    import ctypes
    jobs, checks, keep = [], [], []
    for K in (128, 16):
        d = make(cuda_dev, [40], torch.float32, 2, 2, K, 16, seed=K)
        o, fin = torch.empty(40, 2, 16, device=cuda_dev), torch.empty(1, 2, 16, K, device=cuda_dev)
        dims, st = ssd.linear_attn_dims((1, 40), 2, 2, K, 16, ssd.SSD_DTYPE_F32), torch.cuda.Stream()
        jobs.append((ssd._lib.ssd_linear_attn_fwd,
                     (d["q"].data_ptr(), d["k"].data_ptr(), d["v"].data_ptr(), d["ld"].data_ptr(), 1.0, d["s0"].data_ptr(), None, None,
                      o.data_ptr(), fin.data_ptr(), None, ctypes.byref(dims), st.cuda_stream)))
        checks.append((o, fin, LO.linattn(d["q"], d["k"], d["v"], d["ld"], 1.0, d["s0"]), K))
        keep.append((d, dims, st))
    torch.cuda.synchronize()
    assert at_once(jobs, 5000) == [0, 0]
    ssd.device_status()
    for o, fin, ref, K in checks:
        check(o, fin, ref, torch.float32, K, 40)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,Hk,K,V", [(4, 4, 128, 128), (4, 2, 8, 120), (2, 1, 40, 24), (6, 2, 96, 72)])
@pytest.mark.parametrize("lens,seg", [([700, 333], 0), ([700, 333], 256), ([1500, 130], 1 << 20), ([32, 7], 0)])
def test_states_and_fp32_outputs_keep_24_bits(ssd, cuda_dev, H, Hk, K, V, dtype, lens, seg):
    """2-norms over each head: the element bounds above count every rounding at its worst and
    against sums without cancellation, and would pass a state kept to 16 bits.
    Tolerance 2^-21 (4.8e-7) of the norm. Inputs of random sign, so that a partial sum of i of n terms
    is sqrt(i / n) of the whole. Tensor cores: 8 products of 16 tokens a chunk, each truncated, 2^-24 of the
    partial sum on average and always towards zero: 2^-24 (sqrt(1/8) + .. + sqrt(8/8)) = 3.4e-7.
    CUDA cores: 64 (chunk) + 128 (scores) roundings of random sign, 2^-24 / sqrt(3) each at most:
    2^-24 sqrt(32 + 64) / sqrt(3) = 3.4e-7. Powers of lam and the sums over at most 12 chunks or 32 tokens,
    2^-24 / sqrt(3) each, add sqrt(14 or 32) of that in the square: 2.0e-7. Together below 4.0e-7. Two bf16 terms of
    w V instead of three would leave 2.7e-6 (2^-8 / sqrt(3) / 1.4, squared)."""
    for decay in ("mixed", -0.01):
        d = make(cuda_dev, lens, dtype, H, Hk, K, V, seed=41, decay=decay)
        ref = LO.linattn(d["q"], d["k"], d["v"], d["ld"], K ** -0.5, d["s0"], lens)
        ssd.set_segment_tokens(seg)
        try:
            o, fin = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["ld"], init_state=d["s0"], cu_seqlens=cu_of(lens, cuda_dev))
        finally:
            ssd.set_segment_tokens(0)
        ssd.device_status()
        rel = lambda x, r, dims: ((x.double() - r).pow(2).sum(dims) / r.pow(2).sum(dims)).sqrt().max().item()  # noqa: E731
        assert rel(fin, ref["final"], (2, 3)) <= 2.0 ** -21
        if dtype == torch.float32:
            assert rel(o, ref["o"], (0, 2)) <= 2.0 ** -21

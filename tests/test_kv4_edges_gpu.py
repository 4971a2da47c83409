"""The key/value step on the GPU where it is easily wrong: scores that jump from one
tile of keys to the next, steps, queries and rows that are not finite, positions
outside the cache, bounds on positions, callers' workspaces, heads in several turns,
and the layers over ragged and captured steps.  Against float64.

Bounds (u = 2^-24; half steps: fp16 2^-11, bf16 2^-8).  A score: fp32 queries in two
fp16 terms 2^-22, 2d products summed with truncation 2d * 2^-23, four factors u, each
of m = max_j sum_i |q_i k_ij| / sqrt(d); its base-2 form y rounds three times, 3 |y| u
ln 2 of e^score.  A weight is off by twice that (its own score and the largest one) and
2^-21 for the exponential and its fp16 terms; bf16 rows take one term, 2^-11, and with
many queries values and keys of 11 bits (2^-11 each: the keys' of m, unless they are
exact) and a cubic for some exponentials, 7.6e-5.  Sums over n keys: 3 n 2^-23.  The
output is within twice the weights' bound of sum_j w_j |v_j|, and 2^-8 (bf16) or 2u of
itself.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from bitlinear_bitnet_quant_b200 import api, build_lib  # noqa: E402
from bitlinear_bitnet_quant_b200 import workloads as wl  # noqa: E402
from oracle import kv4_oracle as KO  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
KERNELS = pytest.mark.parametrize("kernel", [1, 2])
DTYPES = pytest.mark.parametrize("dtype", [F32, BF16])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()
    api.lib()
    yield
    assert api.bitnet_device_error() == 0


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def normal(rng, n, width, dtype, scale=1.0):
    return torch.from_numpy((rng.standard_normal((n, width)) * scale).astype(np.float32)).cuda().to(dtype)


def codes(rng, *shape):
    return np.clip(np.rint(rng.standard_normal(shape) * 2.6), -8, 7).astype(np.int8)


def hold(kc, ks, vc, vs):
    """The cache of codes [B, kv, T, d] and steps [B, kv, T], and the values it stands for."""
    dev = api.KV4Cache(*(torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in
                         (KO.pack_codes(kc), ks.astype(np.float32), KO.pack_codes(vc), vs.astype(np.float32))))
    with np.errstate(invalid="ignore"):              # (a code 0 of an infinite step)
        return dev, *(c * s.astype(np.float32).astype(np.float64)[..., None] for c, s in ((kc, ks), (vc, vs)))


def steps(rng, *shape):
    return rng.uniform(0.1, 0.9, shape)


def check(got, q, k, v, positions, kernel, dtype, window=0, sinks=0, exact_keys=False):
    """got, q [n, heads, d] of one sequence; k, v [kv, T, d]."""
    kv, T, d = k.shape
    heads, bf16, many = q.shape[1], dtype == BF16, kernel != 1 and dtype == BF16
    see = KO.visible(np.where((positions >= 0) & (positions < T), positions, -1), T, window, sinks)
    for h in range(heads):
        ref, wv, m = KO.attention(q[:, h], k[h // (heads // kv)], v[h // (heads // kv)], see)
        E = (2.0 ** -22 + 2 * d * 2.0 ** -23 + 4 * U + (many and not exact_keys) * 2.0 ** -11) * m
        E = E + 3 * (m / math.log(2) + 256) * U * math.log(2)
        w = 2 * E + 2.0 ** -21 + 3 * see.sum(-1) * 2.0 ** -23 + bf16 * 2.0 ** -11 + many * (2.0 ** -11 + 7.6e-5)
        tol = 2 * w[:, None] * wv + (2.0 ** -8 if bf16 else 2 * U) * np.abs(ref) + 1e-30
        err = np.abs(got[:, h] - ref)
        assert np.all(err <= tol), (h, (err / tol).max())


# ------------------------------------------------------- scores that jump --

# The spike's score in base 2 is 16.3 c 2^e and its value step 2^F, the others' scores are near zero: the
# last three pass 2^127 of the maximum so far
@KERNELS
@DTYPES
@pytest.mark.parametrize("c,e,F", [(1, 0, -1), (7, 0, -1), (1, 3, -1), (3, 2, -1), (5, 2, -1), (1, 5, -1), (3, 0, 59),
                                   (1, 2, 59), (7, 5, 59)])
def test_a_score_far_above_the_tiles_before(c, e, F, dtype, kernel):
    """One key of a later tile that carries all the weight, at every place of eight."""
    rng = np.random.default_rng(100 * c + e)
    B, L, T, d = 16, 33, 432, 128
    base = -15 if F > 0 else -1                      # the other value steps
    kc, vc = codes(rng, B, 1, T, d), codes(rng, B, 1, T, d)
    ks, vs = np.full((B, 1, T), 2.0 ** -6), 2.0 ** base * rng.uniform(1, 2, (B, 1, T))
    for b in range(B):
        j = (128 if b < 8 else 312) + b % 8
        kc[b, 0, j], ks[b, 0, j], vs[b, 0, j] = c, 2.0 ** e, 2.0 ** F * 1.5
    vc[vc == 0] = 1                                  # (no output that only the keys of tiny weights make)
    cache, k, v = hold(kc, ks, vc, vs)
    q = torch.ones((B * L, d), dtype=dtype, device="cuda")
    A = host(api.bitnet_kv4_attention(q, cache, B, L, T - L, 1, kernel=kernel)).reshape(B, L, 1, d)
    for b in range(B):
        check(A[b], host(q).reshape(B, L, 1, d)[b], k[b], v[b], T - L + np.arange(L), kernel, dtype, exact_keys=True)


@KERNELS
@DTYPES
@pytest.mark.parametrize("size,window", [(2.0 ** -8, 0), (2.0 ** -4, 0), (2.0 ** -2, 0), (2.0 ** -4, 200)])
def test_scores_that_grow_along_the_keys(size, window, dtype, kernel):
    """Key j's score in base 2 is 16.3 j size: every key carries most of the weight of its own query."""
    rng = np.random.default_rng(7)
    L, T, d = 300, 432, 128
    kc, vc = np.ones((1, 1, T, d), dtype=np.int8), codes(rng, 1, 1, T, d)
    vc[vc == 0] = 1
    cache, k, v = hold(kc, np.arange(T)[None, None] * size, vc, steps(rng, 1, 1, T))
    q = torch.ones((L, d), dtype=dtype, device="cuda")
    A = host(api.bitnet_kv4_attention(q, cache, 1, L, T - L, 1, window=window, sinks=3, kernel=kernel)).reshape(L, 1, d)
    check(A, np.ones((L, 1, d)), k[0], v[0], T - L + np.arange(L), kernel, dtype, window, 3, exact_keys=True)


# ------------------------------------------- what is not finite, by its place --

@KERNELS
@DTYPES
@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("L,t0,j", [(1, 400, 5), (1, 400, 399), (40, 300, 7), (40, 300, 310), (150, 0, 3), (150, 0, 70),
                                    (150, 0, 140)])
def test_a_step_that_is_not_finite(L, t0, j, bad, dtype, kernel):
    """Makes exactly the queries that see its key NaN, in tiles that they see whole and in others."""
    rng = np.random.default_rng(31)
    heads, kv, d, T = 8, 2, 128, 448
    clean = [codes(rng, 1, kv, T, d), steps(rng, 1, kv, T), codes(rng, 1, kv, T, d), steps(rng, 1, kv, T)]
    q = normal(rng, L, heads * d, dtype, 1.5)
    at = t0 + np.arange(L)
    for which in (1, 3):
        parts = [x.copy() for x in clean]
        parts[which][0, :, j] = bad
        cache, k, v = hold(*parts)
        A = host(api.bitnet_kv4_attention(q, cache, 1, L, t0, heads, kernel=kernel)).reshape(L, heads, d)
        assert np.isnan(A[at >= j]).all()
        before = at < j
        if before.any():
            check(A[before], host(q).reshape(L, heads, d)[before], k[0, :, :j], v[0, :, :j], at[before], kernel, dtype)
    # behind the last query the same steps, and negative ones, are not seen
    parts = [x.copy() for x in clean]
    for which in (1, 3):
        parts[which][0, :, t0 + L:] = bad
        parts[which][0, :, t0 + L] = -math.inf
    cache, k, v = hold(*parts)
    A = host(api.bitnet_kv4_attention(q, cache, 1, L, t0, heads, kernel=kernel)).reshape(L, heads, d)
    check(A, host(q).reshape(L, heads, d), k[0, :, :t0 + L], v[0, :, :t0 + L], at, kernel, dtype)


@KERNELS
@DTYPES
@pytest.mark.parametrize("e", [0, 19, 20, 24, 28, 30, 58])
def test_rows_outside_the_cache_are_zero_beside_large_values(e, dtype, kernel):
    """Value steps of 2^e; some of a block's positions before or behind the cache, or at and past the bound."""
    rng = np.random.default_rng(41)
    L, heads, d, T = 150, 2, 64, 160
    cache, k, v = hold(codes(rng, 1, 1, T, d), steps(rng, 1, 1, T), codes(rng, 1, 1, T, d),
                       2.0 ** e * rng.uniform(1, 2, (1, 1, T)))
    q = normal(rng, L, heads * d, dtype, 1.5)
    for first, t_max in ((T - 60, None), (-40, None), (0, 100), (20, 129)):
        A = host(api.bitnet_kv4_attention(q, cache, 1, L, 0, heads, t_max=t_max, pos=ints([first]),
                                          kernel=kernel)).reshape(L, heads, d)
        at = first + np.arange(L)
        inside = (at >= 0) & (at < (t_max or T))
        assert not A[~inside].any() and not np.isnan(A).any()
        check(A[inside], host(q).reshape(L, heads, d)[inside], k[0], v[0], at[inside], kernel, dtype)


@KERNELS
@DTYPES
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_past_the_range_of_fp32(sign, dtype, kernel):
    """Every score of a row past the range, to either side: NaN.  One past the smallest number
    beside finite ones weighs nothing."""
    rng = np.random.default_rng(51)
    T, d = 144, 128
    for L, t0 in ((1, 130), (140, 0)):
        kc, ks = np.full((1, 1, T, d), sign, dtype=np.int8), np.full((1, 1, T), 2.0 ** 59)
        vc, vs = codes(rng, 1, 1, T, d), steps(rng, 1, 1, T)
        q = torch.full((L, d), 1e38, dtype=dtype, device="cuda")
        A = api.bitnet_kv4_attention(q, hold(kc, ks, vc, vs)[0], 1, L, t0, 1, kernel=kernel)
        assert A.isnan().all()
        if sign < 0:                                 # a key whose score is zero
            kc[0, 0, 2] = 0
            cache, k, v = hold(kc, ks * np.where(np.arange(T) == 2, 2.0 ** -59, 1.0), vc, vs)
            A = host(api.bitnet_kv4_attention(q, cache, 1, L, t0, 1, kernel=kernel))
            at = t0 + np.arange(L)
            assert np.isnan(A[at < 2]).all()
            assert np.all(np.abs(A[at >= 2] - v[0, 0, 2]) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(v[0, 0, 2]))


@KERNELS
@DTYPES
def test_an_infinite_query_is_nan(dtype, kernel):
    """Also where every score is -inf."""
    rng = np.random.default_rng(52)
    T, d, heads = 144, 64, 2
    for L, t0 in ((1, 0), (1, 130), (140, 0)):
        kc = codes(rng, 1, 1, T, d)
        kc[..., 9] = -3
        cache, k, v = hold(kc, steps(rng, 1, 1, T), codes(rng, 1, 1, T, d), steps(rng, 1, 1, T))
        for bad in (math.inf, -math.inf):
            q = normal(rng, L, heads * d, dtype)
            q[-1, d + 9] = bad                       # the last token's second head
            A = host(api.bitnet_kv4_attention(q, cache, 1, L, t0, heads, kernel=kernel)).reshape(L, heads, d)
            assert np.isnan(A[-1, 1]).all()
            qh = host(q).reshape(L, heads, d)
            check(A[:, :1], qh[:, :1], k[0], v[0], t0 + np.arange(L), kernel, dtype)
            check(A[:-1, 1:], qh[:-1, 1:], k[0], v[0], t0 + np.arange(L - 1), kernel, dtype)


@pytest.mark.parametrize("dtype,d,norm,had,B,L", [(F32, 128, False, False, 2, 5), (BF16, 64, True, True, 1, 40),
                                                  (BF16, 128, False, True, 2, 700), (F32, 64, True, False, 3, 1)])
def test_append_keeps_what_is_not_finite(dtype, d, norm, had, B, L):
    """A key or value row with a NaN or an infinity is held with the step NaN, reads back as NaN and makes the
    queries that see it NaN; every other row is held as without it."""
    rng = np.random.default_rng(61)
    heads, kv, n = 4, 2, B * L
    q, k, v = (normal(rng, n, w * d, dtype) for w in (heads, kv, kv))
    kw = dict(norm=norm, hadamard=had)
    T = L + 16
    clean, cache = api.bitnet_kv4_cache(B, T, kv, d), api.bitnet_kv4_cache(B, T, kv, d)
    api.bitnet_kv4_append(q, k, v, clean, B, L, 0, heads, **kw)
    bad_k, bad_v = torch.zeros((n, kv), dtype=torch.bool, device="cuda"), torch.zeros((n, kv), dtype=torch.bool, device="cuda")
    for i, (x, seen, val) in enumerate([(k, bad_k, math.nan), (k, bad_k, math.inf), (v, bad_v, math.nan),
                                        (v, bad_v, -math.inf)]):
        r, h = (5 * i + 2) % n, i % kv
        x[r, h * d + 7 * i + 3] = val
        seen[r, h] = True
    Qo = api.bitnet_kv4_append(q, k, v, cache, B, L, 0, heads, **kw)
    K, V = api.bitnet_kv4_read(cache, B, L, 0)
    for bad, got, c, s, c0, s0 in ((bad_k, K, cache.kc, cache.ks, clean.kc, clean.ks),
                                   (bad_v, V, cache.vc, cache.vs, clean.vc, clean.vs)):
        held = bad.view(B, L, kv).transpose(1, 2)
        assert torch.equal(s[:, :, :L].isnan(), held)
        assert torch.equal(got.view(n, kv, d).isnan(), bad[:, :, None].expand(n, kv, d))
        assert torch.equal(c[:, :, :L][~held], c0[:, :, :L][~held]) and torch.equal(s[:, :, :L][~held], s0[:, :, :L][~held])
    sees = (bad_k | bad_v).view(B, L, kv).int().cummax(1).values.bool().repeat_interleave(heads // kv, -1)
    for kernel in (1, 2):
        A = api.bitnet_kv4_attention(Qo, cache, B, L, 0, heads, kernel=kernel).view(B, L, heads, d)
        assert torch.equal(A.isnan(), sees[..., None].expand(B, L, heads, d))


# --------------------------------------- bounds, workspaces, heads in turns --

@KERNELS
@DTYPES
@pytest.mark.parametrize("B,L,ctx,T", [(1, 1, 300, 8192), (2, 70, 500, 2048)])
def test_a_bound_on_the_positions_and_a_callers_workspace(B, L, ctx, T, dtype, kernel):
    """Any bound past the last position gives the attention within its bounds; rows at and past a smaller one are zero.
    A workspace of the size asked for is enough and nothing behind it is written; a byte less is refused."""
    rng = np.random.default_rng(71)
    heads, kv, d = 4, 2, 128
    cache, k, v = hold(codes(rng, B, kv, T, d), steps(rng, B, kv, T), codes(rng, B, kv, T, d), steps(rng, B, kv, T))
    q = normal(rng, B * L, heads * d, dtype, 1.5)
    before = [ctx - 7 * b for b in range(B)]
    for t_max in (ctx + L, ctx + L + 130, T - 1, T, 0):
        need = api.bitnet_kv4_attention_workspace_size(dtype, B, L, heads, kv, d, T, t_max=t_max, kernel=kernel)
        room = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        A = api.bitnet_kv4_attention(q, cache, B, L, 0, heads, t_max=t_max, pos=ints(before), workspace=room[:need],
                                     kernel=kernel)
        assert bool((room[need:] == 0xA5).all())
        for b in range(B):
            check(host(A).reshape(B, L, heads, d)[b], host(q).reshape(B, L, heads, d)[b], k[b], v[b],
                  before[b] + np.arange(L), kernel, dtype)
        own = api.bitnet_kv4_attention(q, cache, B, L, 0, heads, t_max=t_max, pos=ints(before), kernel=kernel)
        assert torch.equal(own, A)
        if need:
            with pytest.raises(api.BitnetError):
                api.bitnet_kv4_attention(q, cache, B, L, 0, heads, t_max=t_max, pos=ints(before),
                                         workspace=room[:need - 1], kernel=kernel)
    A = host(api.bitnet_kv4_attention(q, cache, B, L, 0, heads, t_max=ctx + L - 1, pos=ints(before), kernel=kernel))
    A = A.reshape(B, L, heads, d)
    assert not A[0, -1].any() and A[0, :-1].any(-1).all() and A[1:].any(-1).all()


@DTYPES
def test_heads_in_several_turns(dtype):
    """Ten heads of 65536 keys: more than a workspace of 256 MB holds at once."""
    g = torch.Generator(device="cuda").manual_seed(81)
    rng = np.random.default_rng(81)
    kv, T, d, L = 10, 65536, 128, 20
    one = api.bitnet_kv4_attention_workspace_size(dtype, 1, L, 1, 1, d, T, kernel=2)
    need = api.bitnet_kv4_attention_workspace_size(dtype, 1, L, kv, kv, d, T, kernel=2)
    assert one < need < kv * one and need % one == 0
    half = lambda: (torch.randint(0, 256, (1, kv, T, d // 2), generator=g, device="cuda", dtype=torch.uint8),
                    torch.rand((1, kv, T), generator=g, device="cuda") * 0.2 + 0.1)
    cache = api.KV4Cache(*half(), *half())
    q = normal(rng, L, kv * d, dtype, 1.5)
    A = api.bitnet_kv4_attention(q, cache, 1, L, T - L, kv, kernel=2)
    got, qh = host(A).reshape(L, kv, d), host(q).reshape(L, kv, d)
    turn = need // one
    for h in (0, turn - 1, turn, kv - 1):            # the ends of the turns
        k, v = (KO.unpack_codes(c[0, h].cpu().numpy()) * host(s)[0, h, :, None]
                for c, s in ((cache.kc, cache.ks), (cache.vc, cache.vs)))
        check(got[:, h:h + 1], qh[:, h:h + 1], k[None], v[None], T - L + np.arange(L), 2, dtype)
    # more workspace, fewer turns: the same rows
    room = torch.empty(kv * one, dtype=torch.uint8, device="cuda")
    assert torch.equal(api.bitnet_kv4_attention(q, cache, 1, L, T - L, kv, workspace=room, kernel=2), A)


# ------------------------------------------------------------- the layers --

def _chain(rng, B, L, T, kv_heads, n_layers=1, **att):
    from bitlinear_bitnet_quant_b200 import chain
    H, F, d = 2048, 512, 128
    sizes = dict(q=(H, H), k=(kv_heads * d, H), v=(kv_heads * d, H), o=(H, H), up=(F, H), gate=(F, H), down=(H, F))
    layers = [chain.quantize_layer({n: torch.from_numpy(wl.gaussian(rng, s, 0.02)).cuda() for n, s in sizes.items()})
              for _ in range(n_layers)]
    make = lambda L: chain.BitLinearChain(layers, B * L, H, F, torch.device("cuda"), attention=dict(
        B=B, L=L, T_cap=T, heads=16, kv_bits=4, kv_heads=kv_heads, **att))
    return [make(l) for l in L]


def test_chain_over_a_ragged_step():
    """A padded batch of prompts, then a step of one token behind each: what the caches hold and the attention's
    rows against float64, with the same steps of the chain's own call."""
    rng = np.random.default_rng(91)
    B, L, T, kv, d = 3, 30, 64, 4, 128
    pre, dec = _chain(rng, B, (L, 1), T, kv, window=20, sinks=2, qk_norm=True)
    dec.kv4 = pre.kv4
    new = [30, 11, 1]
    for ch, Ls, pos, lens in ((pre, L, [0] * B, new), (dec, 1, new, [1, 0, 1])):
        x = torch.from_numpy(wl.gaussian(rng, (B * Ls, 2048))).cuda()
        held = [t.clone() for t in ch.kv4[0]]
        out = ch.forward(x, pos=ints(pos), lens=ints(lens))
        for b in range(B):
            assert torch.isfinite(out[b * Ls:b * Ls + lens[b]]).all()
            n = pos[b] + lens[b]
            for t, was in zip(ch.kv4[0], held):      # nothing but the real tokens' rows is written
                assert torch.equal(t[b, :, :pos[b]], was[b, :, :pos[b]]) and torch.equal(t[b, :, n:], was[b, :, n:])
            if not lens[b]:
                continue
            sl = slice(b * Ls, b * Ls + lens[b])
            one = api.KV4Cache(*(t[b:b + 1] for t in ch.kv4[0]))
            K, V = api.bitnet_kv4_read(one, 1, n, 0)
            k, v = (host(t).reshape(n, kv, d).transpose(1, 0, 2) for t in (K, V))
            at = pos[b] + np.arange(lens[b])
            kt = KO.turn_rows(host(ch.k)[sl].reshape(-1, kv, d), at, hadamard=True)
            err = np.abs(k[:, pos[b]:].transpose(1, 0, 2) - kt)
            assert np.all(err <= np.abs(kt).max(-1, keepdims=True) / 14 * 1.0001)
            check(host(ch.att)[sl].reshape(-1, 16, d), host(ch.q)[sl].reshape(-1, 16, d), k, v, at, 0, F32, 20, 2)


def test_a_captured_chain_replays_at_other_positions():
    rng = np.random.default_rng(92)
    B, T, kv = 2, 96, 4
    ch, eager = _chain(rng, B, (1, 1), T, kv, n_layers=2, hadamard=False)
    x = torch.from_numpy(wl.gaussian(rng, (B, 2048))).cuda()
    pos, lens = ints([0, 0]), ints([1, 1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ch.forward(x, stream=s, pos=pos, lens=lens)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = ch.forward(x, stream=s, pos=pos, lens=lens)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(ch.kv4, eager.kv4):
        for t, u in zip(a, b):
            u.copy_(t)
    for at, n in (([1, 1], [1, 1]), ([2, 2], [1, 0]), ([3, 2], [1, 1]), ([90, 40], [1, 1])):
        x.copy_(torch.from_numpy(wl.gaussian(rng, (B, 2048))))
        pos.copy_(ints(at))
        lens.copy_(ints(n))
        graph.replay()
        want = eager.forward(x, pos=ints(at), lens=ints(n))
        real = torch.tensor(n, device="cuda") > 0
        assert torch.equal(out[real], want[real])
        for a, b in zip(ch.kv4, eager.kv4):
            for t, u in zip(a, b):
                assert torch.equal(t, u)


def _kernels_of(call):
    """Kernels that call() enqueues, counted in a capture of it."""
    from cuda.bindings import driver
    call()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    raw = driver.CUgraph(graph.raw_cuda_graph())
    err, _, count = driver.cuGraphGetNodes(raw)
    assert int(err) == 0
    err, nodes, count = driver.cuGraphGetNodes(raw, count)
    assert int(err) == 0 and len(nodes) == count
    kinds = [driver.cuGraphNodeGetType(n) for n in nodes]
    assert all(int(e) == 0 for e, _ in kinds)
    return sum(kind == driver.CUgraphNodeType.CU_GRAPH_NODE_TYPE_KERNEL for _, kind in kinds)


@pytest.mark.parametrize("L,T,t0,kw", [(1, 64, 20, {}), (1, 4096, 4000, {}), (512, 512, 0, {}),
                                       (1, 4096, 0, dict(pos=[5])), (1, 4096, 0, dict(pos=[5], t_max=40))])
def test_launches_counts_the_kernels(L, T, t0, kw):
    rng = np.random.default_rng(93)
    ch, = _chain(rng, 1, (L,), T, 16, n_layers=2)
    x = torch.from_numpy(wl.gaussian(rng, (L, 2048))).cuda()
    kw = dict(kw, pos=ints(kw["pos"])) if "pos" in kw else kw
    assert _kernels_of(lambda: ch.forward(x, t0=t0, **kw)) == ch.launches

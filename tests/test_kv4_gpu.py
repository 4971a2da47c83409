"""The key/value step on the GPU against float64: norms, rotation and append (fp32
and 4-bit caches), the way back to values, and attention over the 4-bit cache.

Bounds (u = 2^-24; half steps: fp16 2^-11, bf16 2^-8):
  turned rows in fp32: the mean of squares is a sum of at most 16 + 3 terms in
    sequence (half of its error in the root), root, quotient, eps, the factor and
    gamma 6 more; cosine and sine round once, the rotation 3 times: 24 u of the
    pair's size; each of log2(d) Hadamard stages and the last factor one more u of
    the row's mean size.
  codes: the kernel's t is within one ulp of the oracle's, so a code may differ only
    where t * s lies within 7 * 2^-22 of a border; steps within 2 ulp.
  attention, fp32: q in two fp16 terms (2^-22 of each value), 2d products summed with
    truncation (2d * 2^-23 of sum |q_i k_i|), four factors of u each: E = (2^-22 +
    2d 2^-23 + 4u) max_j sum_i |q_i k_ij| / sqrt(d) on a score, and its base-2 form,
    below 2^8 here, rounds three times (3 * 2^8 u ln 2); weights: 2 E' + 2^-21 for the
    exponential and the two fp16 terms; sums over n keys and the output's 2n products:
    3 n 2^-23.  An output is then within 2 * that of sum_j w_j |v_j|.
  attention, bf16: the weights' one fp16 term adds 2^-11, the output 2^-8 of itself.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from bitlinear_bitnet_quant_b200 import workloads as wl  # noqa: E402
from oracle import bitnet_oracle as O  # noqa: E402
from oracle import kv4_oracle as KO  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
api = None


@pytest.fixture(scope="module", autouse=True)
def _lib():
    global api
    from bitlinear_bitnet_quant_b200 import api as _api, build_lib
    build_lib.build()
    api = _api
    api.lib()
    yield
    assert api.bitnet_device_error() == 0


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def rows(rng, n, width, dtype, scale=1.0):
    """(device rows, the float64 values they hold)"""
    t = torch.from_numpy((rng.standard_normal((n, width)) * scale).astype(np.float32)).cuda().to(dtype)
    return t, host(t)


F32, BF16 = torch.float32, torch.bfloat16


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append --

#    dtype, B, L, heads, kv, d, rot, norm, had, t0, pos, lens
APPENDS = [
    (F32, 1, 1, 16, 16, 128, 128, True, True, 512, None, None),
    (F32, 32, 1, 16, 16, 128, 128, False, True, 0, "ragged", None),
    (BF16, 2, 37, 8, 2, 128, 128, True, False, 5, None, None),
    (BF16, 3, 50, 5, 1, 64, 32, True, True, 0, "ragged", "ragged"),
    (F32, 2, 700, 3, 3, 64, 64, False, False, 3, None, "ragged"),
    (BF16, 1, 1300, 8, 8, 128, 0, False, True, 0, None, None),
    (F32, 4, 3, 7, 7, 128, 64, True, False, 100000, "ragged", None),
]


def _append_inputs(case, four):
    dtype, B, L, heads, kv, d, rot, norm, had, t0, pos, lens = case
    rng = np.random.default_rng(L * 100 + heads)
    before = [(7 * b + 2) % 13 for b in range(B)] if pos else [0] * B
    new = [L * (b + 1) // B if b % 2 == 0 else max(0, L - 3 * b) for b in range(B)] if lens else [L] * B
    at = np.array([[t0 + before[b] + l for l in range(L)] for b in range(B)])
    real = np.array([[l < new[b] for l in range(L)] for b in range(B)])
    T = -(-(t0 + L + 13) // 16) * 16
    q, q64 = rows(rng, B * L, heads * d, dtype)
    k, k64 = rows(rng, B * L, kv * d, dtype, 2.0)
    v, v64 = rows(rng, B * L, kv * d, dtype)
    gq, gk = (torch.from_numpy(rng.uniform(0.5, 1.5, d).astype(np.float32)).cuda() for _ in range(2))
    kw = dict(pos=ints(before) if pos else None, lens=ints(new) if lens else None, rot_dim=rot)
    n = B * L
    turn = lambda x, h, g, nm, hd: KO.turn_rows(x.reshape(n, h, d), at.reshape(-1), host(g), norm=nm, rot_dim=rot,
                                                hadamard=hd)
    return locals()


def _check_turned(got, ref, x_size, d, had, bf16):
    """x_size: an upper bound on the sizes that the roundings are relative to."""
    tol = (24 * x_size + (had * (math.log2(d) + 1 + 24)) * x_size) * U + (2.0 ** -8 * np.abs(ref) if bf16 else 0)
    err = np.abs(got - ref)
    assert np.all(err <= tol + 1e-30), (err / (tol + 1e-30)).max()


def _sizes(ref, d, had):
    """Pair sizes of turned rows, or with the Hadamard transform the mean size sum |y| / sqrt(d)."""
    if had:
        y = ref @ KO.hadamard_matrix(d)              # back before the transform
        return np.broadcast_to(np.abs(y).sum(-1, keepdims=True) / math.sqrt(d), ref.shape)
    p = np.sqrt((ref.reshape(*ref.shape[:-1], -1, 2) ** 2).sum(-1))
    return 2 * np.repeat(p, 2, axis=-1)


@pytest.mark.parametrize("case", APPENDS)
def test_kv4_append_and_read(case):
    c = _append_inputs(case, True)
    dtype, B, L, heads, kv, d, rot, norm, had, t0 = case[:10]
    cache = api.bitnet_kv4_cache(B, c["T"], kv, d)
    for t in cache:
        t.fill_(85)
    Qo = torch.full((B * L, heads * d), 3.25, device="cuda", dtype=dtype)
    out = api.bitnet_kv4_append(c["q"], c["k"], c["v"], cache, B, L, t0, heads, norm=norm, gamma_q=c["gq"],
                                gamma_k=c["gk"], hadamard=had, Qo=Qo, **c["kw"])
    assert out is Qo
    real, at = c["real"], c["at"]
    q_ref = c["turn"](c["q64"], heads, c["gq"], norm, had).reshape(B, L, heads, d)
    got = host(Qo).reshape(B, L, heads, d)
    _check_turned(got[real], q_ref[real], _sizes(q_ref[real], d, had), d, had, dtype == BF16)
    assert np.all(got[~real] == 3.25)                # padding is left as it was
    k_ref = c["turn"](c["k64"], kv, c["gk"], norm, had).reshape(B, L, kv, d)
    v_ref = c["v64"].reshape(B, L, kv, d)
    Kr = torch.full((B * L, kv * d), 9.0, device="cuda")
    Vr = torch.full((B * L, kv * d), 9.0, device="cuda")
    api.bitnet_kv4_read(cache, B, L, t0, pos=c["kw"]["pos"], lens=c["kw"]["lens"], K=Kr, V=Vr)
    b16 = api.bitnet_kv4_read(cache, B, L, t0, pos=c["kw"]["pos"], lens=c["kw"]["lens"], dtype=BF16)
    for ref, codes, steps, read, read16 in ((k_ref, cache.kc, cache.ks, Kr, b16[0]), (v_ref, cache.vc, cache.vs, Vr, b16[1])):
        codes, steps = codes.cpu().numpy(), steps.cpu().numpy()
        want, step, z = KO.hold_rows(ref)
        written = np.zeros((B, c["T"]), dtype=bool)
        for b, l in zip(*np.nonzero(real)):
            p = at[b, l]
            written[b, p] = True
            have = KO.unpack_codes(codes[b, :, p])
            near = np.abs(z[b, l] - np.floor(z[b, l]) - 0.5) < 7 * 2.0 ** -22
            assert np.all((have == want[b, l]) | (near & (np.abs(have - want[b, l]) <= 1)))
            assert np.all(np.abs(steps[b, :, p] - step[b, l]) <= 2.0 ** -22 * step[b, l])
            held = have.astype(np.float32) * steps[b, :, p][:, None]
            assert np.array_equal(host(read[b * L + l]), held.reshape(-1).astype(np.float64))
            assert torch.equal(read16[b * L + l].cpu(), torch.from_numpy(held.reshape(-1)).to(BF16))
        # rows outside the step are untouched, padding is not read
        keep = ~written[:, None, :].repeat(kv, 1)
        assert np.all(codes[keep] == 85) and np.all(steps[keep] == 85)
        flat = real.reshape(-1)
        assert np.all(host(read)[~flat] == 9.0) and not read16.float().cpu().numpy()[~flat].any()


@pytest.mark.parametrize("case", APPENDS)
def test_qk_norm_rope_append(case):
    c = _append_inputs(case, False)
    dtype, B, L, heads, kv, d, rot, _, _, t0 = case[:10]
    T = c["T"]
    Kc = torch.full((B, T, kv * d), 7.5, device="cuda")
    Vc = Kc.clone()
    Qo = api.bitnet_qk_norm_rope_append(c["q"], c["k"], c["v"], Kc, Vc, B, L, t0, heads, kv_heads=kv, gamma_q=c["gq"],
                                        gamma_k=c["gk"], **c["kw"])
    assert Qo.dtype == F32
    real, at = c["real"], c["at"]
    q_ref = c["turn"](c["q64"], heads, c["gq"], True, False).reshape(B, L, heads, d)
    _check_turned(host(Qo).reshape(B, L, heads, d)[real], q_ref[real], _sizes(q_ref[real], d, False), d, 0, False)
    k_ref = c["turn"](c["k64"], kv, c["gk"], True, False).reshape(B, L, kv, d)
    kh, vh = host(Kc).reshape(B, T, kv, d), host(Vc).reshape(B, T, kv, d)
    written = np.zeros((B, T), dtype=bool)
    bs, ls = np.nonzero(real)
    written[bs, at[bs, ls]] = True
    k_got = kh[bs, at[bs, ls]]
    _check_turned(k_got, k_ref[bs, ls], _sizes(k_ref[bs, ls], d, False), d, 0, False)
    assert np.array_equal(vh[bs, at[bs, ls]], c["v64"].reshape(B, L, kv, d)[bs, ls])
    assert np.all(kh[~written] == 7.5) and np.all(vh[~written] == 7.5)
    if dtype == F32:                                 # in place
        again = c["q"].clone()
        assert api.bitnet_qk_norm_rope_append(again, c["k"], c["v"], Kc, Vc, B, L, t0, heads, kv_heads=kv,
                                              gamma_q=c["gq"], gamma_k=c["gk"], Qo=again, **c["kw"]) is again
        keep = torch.from_numpy(real.reshape(-1)).cuda()
        assert torch.equal(again[keep], Qo[keep]) and torch.equal(again[~keep], c["q"][~keep])


def test_append_reads_views_of_one_projection():
    """Q, K and V as column ranges of one tensor give what dense copies give."""
    rng = np.random.default_rng(3)
    B, L, heads, kv, d = 2, 9, 6, 2, 128
    qkv, _ = rows(rng, B * L, (heads + 2 * kv) * d, BF16)
    q, k, v = qkv[:, :heads * d], qkv[:, heads * d:(heads + kv) * d], qkv[:, (heads + kv) * d:]
    outs = []
    for parts in ((q, k, v), tuple(x.contiguous() for x in (q, k, v))):
        cache = api.bitnet_kv4_cache(B, 16, kv, d)
        outs.append((api.bitnet_kv4_append(*parts, cache, B, L, 2, heads, norm=True, hadamard=True), *cache))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_append_edge_rows():
    """Zero rows, a single spike, tiny rows; a row outside the cache is turned but not appended."""
    d, T = 128, 16
    x = torch.zeros((4, d), device="cuda")
    x[1, 5] = -3.0
    x[2] = 1e-7
    x[3] = torch.linspace(-1, 1, d, device="cuda")
    cache = api.bitnet_kv4_cache(1, T, 1, d)
    out = api.bitnet_kv4_append(x, x, x, cache, 1, 4, 0, 1, rot_dim=0, pos=ints([14]))
    assert torch.equal(out, x)                       # no norm, no rotation: as it was
    codes = KO.unpack_codes(cache.kc.cpu().numpy())[0, 0]
    want, step, _ = KO.hold_rows(host(x))
    assert np.array_equal(codes[14:16], want[:2]) and not codes[:14].any()
    assert np.array_equal(cache.ks.cpu().numpy()[0, 0, 14:], step[:2])
    assert codes[15, 5] == -7 and np.count_nonzero(codes) == 1
    neg = api.bitnet_kv4_cache(1, T, 1, d)
    api.bitnet_kv4_append(x, x, x, neg, 1, 4, 0, 1, rot_dim=0, pos=ints([-2]))
    codes = KO.unpack_codes(neg.vc.cpu().numpy())[0, 0]
    assert np.array_equal(codes[:2], want[2:]) and not codes[2:].any()


# --------------------------------------------------------------- attention --

def _cache(rng, B, kv, T, d, spread=1.0):
    codes = lambda: np.clip(np.rint(rng.standard_normal((B, kv, T, d)) * 2.6), -8, 7).astype(np.int8)
    steps = lambda: (0.3 * np.exp(spread * rng.uniform(-1, 1, (B, kv, T)))).astype(np.float32)
    kc, vc, ks, vs = codes(), codes(), steps(), steps()
    dev = api.KV4Cache(*(torch.from_numpy(x).cuda() for x in (KO.pack_codes(kc), ks, KO.pack_codes(vc), vs)))
    return dev, kc * ks[..., None].astype(np.float64), vc * vs[..., None].astype(np.float64)


def _check_attention(got, q, k, v, positions, heads, window, sinks, bf16):
    """got, q [n, heads, d] of one sequence; k, v [kv, T, d]."""
    kv, T, d = k.shape
    see = KO.visible(np.where((positions >= 0) & (positions < T), positions, -1), T, window, sinks)
    for h in range(heads):
        kvh = h // (heads // kv)
        ref, wv, mag = KO.attention(q[:, h], k[kvh], v[kvh], see)
        n = see.sum(-1)
        E = (2.0 ** -22 + 2 * d * 2.0 ** -23 + 4 * U) * mag + 3 * 256 * U * math.log(2)
        w = 2 * E + 2.0 ** -21 + 3 * n * 2.0 ** -23 + (2.0 ** -11 if bf16 else 0)
        tol = 2 * w[:, None] * wv + (2.0 ** -8 if bf16 else 2 * U) * np.abs(ref) + 1e-30
        err = np.abs(got[:, h] - ref)
        assert np.all(err <= tol), (h, (err / tol).max())


#    dtype, B, L, ctx, heads, kv, d, window, sinks, pos, lens
ATTENTIONS = [
    (F32, 1, 1, 0, 1, 1, 128, 0, 0, None, None),
    (F32, 2, 1, 40, 16, 16, 128, 0, 0, None, None),
    (F32, 32, 1, 512, 4, 4, 128, 0, 0, None, None),
    (BF16, 3, 1, 1999, 8, 2, 128, 0, 0, "ragged", None),
    (BF16, 1, 1, 9000, 8, 1, 64, 0, 0, None, None),
    (F32, 2, 3, 77, 6, 2, 64, 0, 0, "ragged", None),
    (F32, 1, 5, 31, 9, 3, 128, 0, 0, None, None),
    (BF16, 2, 2, 600, 10, 2, 128, 100, 3, "ragged", "ragged"),
    (F32, 1, 1, 700, 2, 1, 128, 1, 0, None, None),
    (F32, 1, 1, 700, 2, 1, 64, 64, 200, None, None),
    (F32, 1, 64, 0, 2, 2, 128, 0, 0, None, None),
    (F32, 2, 130, 70, 4, 2, 128, 0, 0, None, "ragged"),
    (BF16, 1, 257, 0, 3, 1, 128, 0, 0, None, None),
    (BF16, 2, 300, 33, 8, 2, 64, 50, 5, "ragged", "ragged"),
    (F32, 1, 400, 200, 5, 1, 64, 128, 130, None, None),
    (F32, 3, 100, 0, 2, 1, 128, 7, 0, "ragged", "ragged"),
    (BF16, 2, 513, 1000, 4, 4, 128, 0, 0, None, None),
    (F32, 1, 129, 2047, 2, 2, 128, 1000, 4, None, None),
    (BF16, 1, 1024, 0, 2, 1, 128, 0, 0, None, None),
    (F32, 1, 700, 0, 3, 1, 128, 0, 0, None, None),
    (F32, 1, 5, 6000, 6, 2, 128, 0, 0, None, None),
    (BF16, 2, 2, 5000, 8, 2, 64, 3000, 7, "ragged", None),
    (F32, 1, 1, 3000, 2, 2, 64, 0, 0, None, None),
]


def _attention_inputs(case, seed=0):
    dtype, B, L, ctx, heads, kv, d, window, sinks, pos, lens = case
    rng = np.random.default_rng(B * 1000 + L * 10 + ctx + seed)
    T = -(-(ctx + L + 5) // 16) * 16
    cache, k, v = _cache(rng, B, kv, T, d)
    q, q64 = rows(rng, B * L, heads * d, dtype, 1.5)
    before = [ctx * (b + 1) // B for b in range(B)] if pos else [ctx] * B
    new = [max(1, L * (B - b) // B) for b in range(B)] if lens else [L] * B
    # what no query sees may hold anything: codes and steps behind the last token and before the window
    for b in range(B):
        see = KO.visible(np.arange(before[b], before[b] + new[b]), T, window, sinks).any(0)
        hide = torch.from_numpy(~see).cuda()
        for codes, steps in ((cache.kc, cache.ks), (cache.vc, cache.vs)):
            codes[b][:, hide] = 0x88
            steps[b][:, hide] = math.nan
        k[b][:, ~see], v[b][:, ~see] = 0.0, 0.0
    return dict(cache=cache, k=k, v=v, q=q, q64=q64, before=before, new=new, pos=ints(before) if pos else None,
                lens=ints(new) if lens else None, t0=0 if pos else ctx)


@pytest.mark.parametrize("kernel", [0, 1, 2])
@pytest.mark.parametrize("case", ATTENTIONS)
def test_kv4_attention(case, kernel):
    """Every case through the kernel for few queries, those for many, and the automatic choice."""
    dtype, B, L, ctx, heads, kv, d, window, sinks, pos, lens = case
    c = _attention_inputs(case)
    A = torch.full((B * L, heads * d), 5.5, dtype=dtype, device="cuda")
    kw = dict(window=window, sinks=sinks, pos=c["pos"], lens=c["lens"], kernel=kernel)
    out = api.bitnet_kv4_attention(c["q"], c["cache"], B, L, c["t0"], heads, A=A, **kw)
    assert out is A
    got, q = host(A).reshape(B, L, heads, d), c["q64"].reshape(B, L, heads, d)
    for b in range(B):
        n = c["new"][b]
        _check_attention(got[b, :n], q[b, :n], c["k"][b], c["v"][b], np.arange(c["before"][b], c["before"][b] + n), heads,
                         window, sinks, dtype == BF16)
        assert np.all(got[b, n:] == 5.5)             # padding is left as it was
    # the same call again, in place, gives the same bits; so does any bound on the positions
    again = c["q"].clone()
    api.bitnet_kv4_attention(again, c["cache"], B, L, c["t0"], heads, A=again, **kw)
    real = torch.tensor([l < c["new"][b] for b in range(B) for l in range(L)], device="cuda")
    assert torch.equal(again[real], A[real]) and torch.equal(again[~real], c["q"][~real])


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("L,heads", [(6, 2), (150, 1)])
def test_kv4_attention_hidden_values_do_not_leak(L, heads, kernel):
    """A query whose tile holds a later token's NaN steps, infinite queries beside it
    and rows outside the cache."""
    rng = np.random.default_rng(11)
    for dtype in (F32, BF16):
        T, d = 160, 128
        cache, k, v = _cache(rng, 1, 1, T, d)
        q, q64 = rows(rng, L, heads * d, dtype)
        cache.ks[0, 0, L - 1] = math.nan             # seen by the last token alone
        cache.vs[0, 0, L - 1] = math.nan
        q[2, 0] = math.inf                           # one head row of token 2
        q[3, 1] = math.nan
        q[4] *= 1e30                                 # and a huge row: the others keep their precision
        A = api.bitnet_kv4_attention(q, cache, 1, L, 0, heads, kernel=kernel)
        keep = [l for l in range(L - 1) if l not in (2, 3, 4)]
        got = host(A).reshape(L, heads, d)
        _check_attention(got[keep], q64.reshape(L, heads, d)[keep], np.nan_to_num(k[0]), np.nan_to_num(v[0]),
                         np.array(keep), heads, 0, 0, dtype == BF16)
        assert np.isnan(got[L - 1]).all()
        if heads > 1:                                # the other heads of tokens 2 and 3
            for l in (2, 3):
                _check_attention(got[l:l + 1, 1:], q64.reshape(L, heads, d)[l:l + 1, 1:], k[0], v[0], np.array([l]), 1, 0,
                                 0, dtype == BF16)
        # a NaN key makes exactly the queries that see it NaN, wherever it lies in its tile
        for j in (0, 3, 6, 7, 13, 33, 70, 127):
            if j < L - 1:
                one, _, _ = _cache(rng, 1, 1, T, d)
                (one.vs if j % 2 else one.ks)[0, 0, j] = math.nan
                A = api.bitnet_kv4_attention(rows(rng, L, heads * d, dtype)[0], one, 1, L, 0, heads, kernel=kernel)
                assert torch.equal(A.isnan().all(-1), torch.arange(L, device="cuda") >= j)
                assert torch.equal(A.isnan().any(-1), torch.arange(L, device="cuda") >= j)
        # a query that sees NaN keys alone
        cache.ks[0, 0, :2] = math.nan
        A = api.bitnet_kv4_attention(rows(rng, L, heads * d, dtype)[0], cache, 1, L, 0, heads, kernel=kernel)
        assert A[:2].isnan().all()
        # every position outside the cache: zeros; some outside: those
        for first, zero in ((T, range(L)), (-L, range(L)), (T - 3, range(3, L)), (-2, range(2))):
            clean = rows(rng, L, heads * d, dtype)[0]
            A = api.bitnet_kv4_attention(clean, api.KV4Cache(*(torch.nan_to_num(t) if t.is_floating_point() else t
                                                               for t in cache)), 1, L, 0, heads, pos=ints([first]), kernel=kernel)
            z = (A == 0).all(-1).cpu().numpy()
            assert np.array_equal(np.nonzero(z)[0], np.array(list(zero)))


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_kv4_attention_rows_that_are_not_finite(dtype, kernel):
    """Queries, and whole blocks of keys, that are not finite make their rows NaN and no others."""
    rng = np.random.default_rng(23)
    L, heads, d, T = 300, 2, 64, 304
    at = np.arange(L)
    for nan_keys in (False, True):
        cache, k, v = _cache(rng, 1, 1, T, d)
        q, q64 = rows(rng, L, heads * d, dtype, 1.5)
        if nan_keys:                                     # keys 128 .. 255, a whole tile
            cache.ks[:, :, 128:256] = math.nan
            bad = at >= 128
        else:
            q[5], q[200], q[250, ::d] = math.nan, math.nan, math.inf
            bad = np.isin(at, (5, 200, 250))
        A = host(api.bitnet_kv4_attention(q, cache, 1, L, 0, heads, kernel=kernel)).reshape(L, heads, d)
        assert np.isnan(A[bad]).all()
        _check_attention(A[~bad], q64.reshape(L, heads, d)[~bad], k[0], v[0], at[~bad], heads, 0, 0, dtype == BF16)
    # scores past the range of fp32, zeros among them
    cache.ks.fill_(2.0 ** 59)
    cache.kc[:, :, ::2] = 0
    A = api.bitnet_kv4_attention(torch.full_like(q, 1e38), cache, 1, L, 0, heads, kernel=kernel)
    assert A.shape == q.shape and api.bitnet_device_error() == 0


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_kv4_attention_wide_steps(dtype, kernel):
    """Value steps over 40 powers of ten, a zero step among them, and scores that
    grow along the keys: the sum of the weights keeps its keys."""
    rng = np.random.default_rng(5)
    for L, T in ((1, 96), (140, 160)):
        heads, d = 2, 128
        cache, k, v = _cache(rng, 1, 1, T, d)
        steps = (10.0 ** rng.uniform(-20, 20, T)).astype(np.float32)
        steps[3] = 0.0
        cache.vs[0, 0] = torch.from_numpy(steps).cuda()
        v = KO.unpack_codes(cache.vc.cpu().numpy()).astype(np.float64) * steps.astype(np.float64)[:, None]
        q, q64 = rows(rng, L, heads * d, dtype, 1.5)
        t0 = T - L
        A = api.bitnet_kv4_attention(q, cache, 1, L, t0, heads, kernel=kernel)
        _check_attention(host(A).reshape(L, heads, d), q64.reshape(L, heads, d), k[0], v[0], t0 + np.arange(L), heads, 0,
                         0, dtype == BF16)


@pytest.mark.parametrize("kernel", [1, 2])
def test_zero_steps_keep_their_weight(kernel):
    """Keys with a zero value step count in the softmax sum."""
    d, T = 128, 32
    cache = api.bitnet_kv4_cache(1, T, 1, d)         # all codes and steps zero: equal weights
    cache.vc[0, 0, 7] = 0x11
    cache.vs[0, 0, 7] = 1.0
    for L in (1, 32):
        q = torch.ones((L, d), device="cuda")
        A = host(api.bitnet_kv4_attention(q, cache, 1, L, T - L, 1, kernel=kernel))
        n = T - L + 1 + np.arange(L)
        ref = np.where(n > 7, 1.0 / n, 0.0)[:, None]
        assert np.all(np.abs(A - ref) <= 2.0 ** -20 * ref)


# ------------------------------------------------------------ whole steps --

def test_captured_step_replays_at_other_positions():
    """Append and attention captured once on another stream, replayed with new rows,
    positions and lengths: what eager calls give."""
    rng = np.random.default_rng(9)
    B, L, heads, kv, d, T = 3, 2, 8, 2, 128, 512
    cache, _, _ = _cache(rng, B, kv, T, d)
    mirror = api.KV4Cache(*(t.clone() for t in cache))
    fresh = lambda: [rows(rng, B * L, w * d, BF16)[0] for w in (heads, kv, kv)]
    q, k, v = fresh()
    pos, lens = ints([0, 5, 9]), ints([2, 2, 1])
    Qo, A = torch.zeros_like(q), torch.zeros_like(q)

    def step(q, k, v, cache, pos, lens, Qo, A):
        api.bitnet_kv4_append(q, k, v, cache, B, L, 0, heads, norm=True, hadamard=True, pos=pos, lens=lens, Qo=Qo)
        api.bitnet_kv4_attention(Qo, cache, B, L, 0, heads, window=100, sinks=2, pos=pos, lens=lens, A=A)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(q, k, v, cache, pos, lens, Qo, A)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step(q, k, v, cache, pos, lens, Qo, A)
    torch.cuda.current_stream().wait_stream(s)
    step(q, k, v, mirror, pos, lens, Qo.clone(), A.clone())
    for first, n in (([100, 200, 300], [2, 1, 2]), ([101, 202, 510], [1, 2, 2])):
        for t, new in zip((q, k, v), fresh()):
            t.copy_(new)
        pos.copy_(ints(first))
        lens.copy_(ints(n))
        A.zero_()
        graph.replay()
        Qe, Ae = torch.zeros_like(q), torch.zeros_like(q)
        step(q, k, v, mirror, pos, lens, Qe, Ae)
        torch.cuda.synchronize()
        assert torch.equal(A, Ae)
        for a, b in zip(cache, mirror):
            assert torch.equal(a, b)


def test_refusals():
    cache = api.bitnet_kv4_cache(2, 64, 2, 128)
    q, kv = torch.zeros((4, 512), device="cuda"), torch.zeros((4, 256), device="cuda")
    ok = dict(B=2, L=2, t0=0, heads=4)
    api.bitnet_kv4_append(q, kv, kv, cache, **ok)
    for err, call in [
        (ValueError, lambda: api.bitnet_kv4_append(q[:3], kv, kv, cache, **ok)),
        (ValueError, lambda: api.bitnet_kv4_append(q, kv[:, :128], kv, cache, **ok)),
        (ValueError, lambda: api.bitnet_kv4_append(q.t().contiguous().t(), kv, kv, cache, **ok)),
        (TypeError, lambda: api.bitnet_kv4_append(q, kv.bfloat16(), kv, cache, **ok)),
        (TypeError, lambda: api.bitnet_kv4_append(q.half(), kv.half(), kv.half(), cache, **ok)),
        (TypeError, lambda: api.bitnet_kv4_append(q, kv, kv, cache, pos=torch.zeros(2, device="cuda"), **ok)),
        (ValueError, lambda: api.bitnet_kv4_append(q, kv, kv, cache, lens=ints([1]), **ok)),
        (ValueError, lambda: api.bitnet_kv4_append(q, kv, kv, cache, gamma_q=torch.ones(64, device="cuda"), **ok)),
        (ValueError, lambda: api.bitnet_kv4_append(q, kv, kv, cache, pos=torch.zeros(2, dtype=torch.int32), **ok)),
        (api.BitnetError, lambda: api.bitnet_kv4_append(q, kv, kv, cache, 2, 2, 63, 4)),
        (api.BitnetError, lambda: api.bitnet_kv4_append(q, kv, kv, cache, rot_dim=3, **ok)),
        (ValueError, lambda: api.bitnet_kv4_attention(q[:, :256], cache, **ok)),
        (TypeError, lambda: api.bitnet_kv4_attention(q, cache, A=torch.zeros_like(q).bfloat16(), **ok)),
        (api.BitnetError, lambda: api.bitnet_kv4_attention(q, cache, window=-1, **ok)),
        (api.BitnetError, lambda: api.bitnet_kv4_attention(q[:, :384].contiguous(), cache, 2, 2, 0, 3)),
        (ValueError, lambda: api.bitnet_kv4_read(cache, 2, 2, 0, K=torch.zeros((4, 128), device="cuda"))),
        (ValueError, lambda: api.bitnet_kv4_read(cache._replace(vs=cache.vs[:, :, :32]), 2, 2, 0)),
    ]:
        with pytest.raises(err):
            call()


@pytest.mark.parametrize("kv_heads,window,qk_norm", [(16, 0, False), (4, 20, True)])
def test_chain_with_4_bit_cache(kv_heads, window, qk_norm):
    """Two layers of the stacked chain (hidden 512, 4 heads of 128) over 4-bit caches: a
    24-token prefill of 2 sequences, then a decode step.  Layer by layer, the rows the
    cache holds and the attention output against float64."""
    from bitlinear_bitnet_quant_b200 import chain
    H, F, d = 2048, 512, 128
    heads = 16
    sizes = dict(q=(H, H), k=(kv_heads * d, H), v=(kv_heads * d, H), o=(H, H), up=(F, H), gate=(F, H), down=(H, F))
    rng = np.random.default_rng(21)
    layers = [chain.quantize_layer({n: torch.from_numpy(wl.gaussian(rng, s, 0.02)).cuda() for n, s in sizes.items()})
              for _ in range(2)]
    B, L = 2, 24
    att = dict(B=B, T_cap=40, heads=heads, kv_bits=4, kv_heads=kv_heads, window=window, sinks=2 if window else 0,
               qk_norm=qk_norm)
    pre = chain.BitLinearChain(layers, B * L, H, F, torch.device("cuda"), attention=dict(att, L=L))
    dec = chain.BitLinearChain(layers, B, H, F, torch.device("cuda"), attention=dict(att, L=1))
    dec.kv4 = pre.kv4
    for ch, x0, t0, Ls in ((pre, wl.gaussian(rng, (B * L, H)), 0, L), (dec, wl.gaussian(rng, (B, H)), L, 1)):
        out = ch.forward(torch.from_numpy(x0).cuda(), t0=t0)
        assert torch.isfinite(out).all()
        ch.t0 = t0
        parts = (torch.from_numpy(x0).cuda(),)
        for li, w in enumerate(layers):
            parts = ch.layer(parts, w, None, li)
            n = t0 + Ls
            K, V = api.bitnet_kv4_read(ch.kv4[li], B, n, 0)
            k, v = (host(x).reshape(B, n, kv_heads, d).transpose(0, 2, 1, 3) for x in (K, V))
            at = np.tile(t0 + np.arange(Ls), B)
            kt = KO.turn_rows(host(ch.k).reshape(-1, kv_heads, d), at, norm=qk_norm, hadamard=True)
            # a held key is within half a step, and the largest |t| is 7 steps
            err = np.abs(k[:, :, t0:].transpose(0, 2, 1, 3).reshape(kt.shape) - kt)
            assert np.all(err <= np.abs(kt).max(-1, keepdims=True) / 14 * 1.0001)
            for b in range(B):
                sl = slice(b * Ls, (b + 1) * Ls)
                _check_attention(host(ch.att)[sl].reshape(Ls, heads, d), host(ch.q)[sl].reshape(Ls, heads, d), k[b], v[b],
                                 t0 + np.arange(Ls), heads, window, 2 if window else 0, False)
    assert pre.launches == 10 * 2 + 1


def test_chain_with_norms_over_the_fp32_cache():
    """qk_norm with the fp32 cache: a one-token context returns V whatever the norms
    are, and a longer one follows float64 within the fp32 attention's bound."""
    from bitlinear_bitnet_quant_b200 import chain
    rng = np.random.default_rng(22)
    H, F, heads, d = 256, 512, 2, 128
    sizes = dict(q=(H, H), k=(H, H), v=(H, H), o=(H, H), up=(F, H), gate=(F, H), down=(H, F))
    layers = [chain.quantize_layer({n: torch.from_numpy(wl.gaussian(rng, s, 0.02)).cuda() for n, s in sizes.items()})]
    g = torch.from_numpy(rng.uniform(0.5, 1.5, d).astype(np.float32)).cuda()
    L = 20
    ch = chain.BitLinearChain(layers, L, H, F, torch.device("cuda"),
                              attention=dict(B=1, L=L, T_cap=L, heads=heads, qk_norm=True, gamma_q=[g], gamma_k=[g]))
    ch.layer((torch.from_numpy(wl.gaussian(rng, (L, H))).cuda(),), layers[0], None, 0)
    assert np.array_equal(host(ch.att)[0], host(ch.v)[0])
    kt = KO.turn_rows(host(ch.k).reshape(L, heads, d), np.arange(L), host(g))
    _check_turned(host(ch.kc[0])[0].reshape(L, heads, d), kt, _sizes(kt, d, False), d, 0, False)
    q, k, v = host(ch.q), host(ch.kc[0])[0], host(ch.v)
    ref = O.attention_f64(q, k, v, heads, O.causal_mask(L, L, 0))
    # scores of 128 fp32 terms: 131 u of sum |q k| / sqrt(d) <= |q| |k| / sqrt(d) <= sqrt(d) max(g)^2; then 2 E + (8 + 2n) u
    tol = (2 * 131 * U * math.sqrt(d) * 1.5 ** 2 + (8 + 2 * L) * U) * np.abs(v).max()
    assert np.abs(host(ch.att) - ref).max() <= tol

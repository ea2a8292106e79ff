"""The 8-bit output head where it can go wrong: values halfway between two codes, products of several
tiles a CTA."""
import ctypes

import numpy as np
import pytest
import torch

from canvas_sampler_gb300 import _lib as C
from canvas_sampler_gb300 import head
from oracle import head as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------------------------- codes
def quotients(y, fmt, block_rows):
    """y / scale in 64 bits as y F / max, which is exact where it lies halfway between two codes."""
    R, C = y.shape
    m = np.empty_like(y)
    for i in range(0, R, block_rows):
        for j in range(0, C, 128):
            at = np.s_[i:i + block_rows, j:j + 128]
            m[at] = max(np.abs(y[at]).max(), O.TINY)
    return y * O.FORMATS[fmt][2] / m


def ties(v, fmt):
    """How many of v lie exactly halfway between two codes."""
    x = np.abs(v) / O.fp8_step(v, fmt)
    return int(np.sum(x - np.floor(x) == 0.5))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_codes_of_a_matrix_are_those_of_the_quotient(dt, block_rows, fmt):
    """The quotient is known to 2^-44, so its fp32 rounding, and with it the code, is the definition's
    unless the quotient lies within 2^-44 of the middle between two fp32 numbers: none of these do."""
    g = gen(31)
    for R, C, shift in ((512, 2816, 0), (200, 1111, 1)):
        buf = (torch.randn(R * C + shift, device="cuda", generator=g) / 16).to(DT[dt])
        x = buf[shift:].view(R, C)
        x[3] = x[3] * 2.0 ** 20
        x[5] = 0
        x[128:256, 128:256] *= 2.0 ** -80
        q, s = head.quantize_fp8(x, block_rows=block_rows, fp8=fmt)
        v = quotients(f64(x), fmt, block_rows)
        assert dt == "fp32" or C != 2816 or ties(v, fmt) > 20  # what this is about
        assert np.array_equal(f64(q), O.fp8_round(v.astype(np.float32), fmt))
        half = 2.0 ** -24  # the scale is one division
        want = O.block_scales(f64(x), fmt, block_rows)
        assert np.all(np.abs(f64(s) - want) <= half * want)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("R,d", [(256, 2816), (40, 5000), (33, 515), (7, 8200)])
def test_codes_of_a_norm_see_one_rounding(dt, fmt, R, d):
    """1 / sqrt(mean + eps) divides out of y / scale. What is left is h (offset + w), rounded to fp32
    once (2^-24 of it, in the element and in the block's maximum), and the quotient's own rounding
    (2^-24): codes are those of the quotient moved by no more than 3 2^-24, and of the quotient itself
    where the product is exact (two bf16 factors)."""
    g = gen(R + d)
    x = torch.randn(R, d, device="cuda", generator=g).to(DT[dt])
    res = (4 * torch.randn(R, d, device="cuda", generator=g)).to(DT[dt])
    for off, scale in ((0.0, 1.0), (1.0, 0.2)):
        w = (scale * torch.randn(d, device="cuda", generator=g)).to(DT[dt])
        q, s, h = head.rmsnorm_fp8(x, w, res, weight_offset=off, fp8=fmt)
        got, v = f64(q), quotients(f64(h) * (off + f64(w)), fmt, 1)
        if dt == "bf16" and off == 0.0:
            assert np.array_equal(got, O.fp8_round(v.astype(np.float32), fmt))
        slack = 1 + 3 * 2.0 ** -24
        a, b = O.fp8_round(v / slack, fmt), O.fp8_round(v * slack, fmt)
        assert np.all((got == a) | (got == b))
        assert np.mean(a != b) < 1e-2  # nearly every code is pinned to one value (ties to two)


# ------------------------------------------------------------------------------------- product
def operands(m, n, k, seed):
    """Codes and scales of an A [m, k] and a B [n, k]."""
    g = gen(seed)
    cols = -(-k // 16) * 16
    code = lambda r: (torch.randn(r, cols, device="cuda", generator=g) * 100).clamp(-400, 400).to(  # noqa: E731
        torch.float8_e4m3fn)[:, :k]
    scale = lambda r: torch.exp(torch.randn(r, -(-k // 128), device="cuda", generator=g)) / 100  # noqa: E731
    return code(m), scale(m), code(n), scale(-(-n // 128))


# with 152 SMs: the first five have two and more 64-column tiles a CTA, the next three 128-column
# ones, the last 256-column ones of CTA pairs
@pytest.mark.parametrize("m,n,k", [(300, 6464, 128), (1409, 1600, 128), (20000, 64, 128), (25000, 120, 160),
                                   (640, 7688, 256), (40000, 128, 128), (300, 14000, 128), (1409, 3200, 128),
                                   (1409, 12000, 128)])
def test_products_of_several_tiles_a_cta(m, n, k):
    """The same sums leave in both types: the bf16 product is the fp32 one rounded."""
    for seed in range(3):
        ops = operands(m, n, k, seed)
        full = head.matmul_fp8(*ops, out_dtype="fp32")
        for _ in range(3):
            out = torch.full((m, n), 7.0, dtype=torch.bfloat16, device="cuda")
            assert torch.equal(head.matmul_fp8(*ops, out=out), full.bfloat16())
    # and the fp32 ones are the definition's: sums of 128 products cut to no worse than 2^-23 of their
    # absolute terms each, one addition a block, half a step of the output
    rows = torch.arange(0, m, max(1, m // 50), device="cuda")
    want, mag = O.matmul(f64(ops[0][rows]), f64(ops[1][rows]), f64(ops[2]), f64(ops[3]))
    bound = (128 + ops[1].shape[1]) * 2.0 ** -23 * mag
    assert np.all(np.abs(f64(full[rows]) - want) <= bound + 2.0 ** -24 * (np.abs(want) + bound))
    assert head.head_status() == 0


# ------------------------------------------------------------------------------------- sampling
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("R", [2, 400])
def test_sampling_with_thousands_of_ties_at_the_kth_logit(dt, R):
    """The list overflows, and top-p is a share of the first k tokens, the lowest indices of the tie."""
    V, k = 20011, 50
    g = gen(R)
    logits = torch.randn(R, V, device="cuda", generator=g).clamp(max=0.25)
    logits[:, 7000] = 1.5
    logits = logits.to(DT[dt])
    u = torch.rand(R, device="cuda", generator=g)
    full = lambda v, t=torch.float32: torch.full((R,), v, dtype=t, device="cuda")  # noqa: E731
    for p in (0.77, 0.3):
        token, prob = head.sample_logits(logits, u, top_k=full(k, torch.int32), top_p=full(p))
        for r in range(0, R, max(1, R // 20)):
            want, pw, margin = O.sample_row(f64(logits[r]), float(u[r]), top_k=k,
                                            top_p=float(np.float32(p)))
            assert margin > 2.0 ** -24 and int(token[r]) == want
            assert abs(float(prob[r]) - pw) <= 2.0 ** -20 * pw


def weights(row, T=1.0):
    """(weights, running sums) of a row in 64 bits and more."""
    w = np.exp((row - row.max()) / T)
    return w, np.cumsum(w.astype(np.longdouble))


def check_long_row(row, u, token, prob, keep=None):
    """The token's share of the running sum has u S in it, to 2^-35 of the mass (weights good to 2^-37
    and rounded to whole units, 2^-37 of the mass in all, in the running sum and in S); prob to 2^-20."""
    w, _ = weights(row)
    if keep is not None:
        w = np.where(keep, w, 0.0)
    c = np.cumsum(w.astype(np.longdouble))
    S, goal = c[-1], np.longdouble(np.float32(u)) * c[-1]
    assert w[token] > 0
    assert c[token] - w[token] - goal <= 2.0 ** -35 * S and goal - c[token] <= 2.0 ** -35 * S, \
        (token, float((c[token] - goal) / S))
    assert abs(prob - float(w[token] / S)) <= 2.0 ** -20 * float(w[token] / S)


LONG = 1 << 24
TAILS = {  # a heavy peak and a long tail of light tokens: where the peak stands, the tail's logit, u's
    "first": (0, -26.5, (0.5, 0.99993, 0.99997, 0.99999)),
    "last": (LONG - 1, -26.5, (0.0, 1e-5, 3e-5, 4.7e-5, 0.3)),
    "lighter": (LONG // 3, -31.0, (1e-8, 2e-7, 0.99, 1.0)),
    "flat": (LONG // 2, -10.0, (0.01, 0.4, 0.6, 0.97)),
}


@pytest.mark.parametrize("name", TAILS)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_sampling_keeps_the_mass_of_a_long_light_tail(name, dt):
    at, tail, us = TAILS[name]
    logits = torch.full((len(us), LONG), tail, device="cuda").to(DT[dt])
    logits[:, at] = 0
    u = torch.tensor(us, device="cuda")
    row = f64(logits[0])
    f = lambda v, t=torch.float32: torch.full((len(us),), v, dtype=t, device="cuda")  # noqa: E731
    order = np.concatenate([[at], np.delete(np.arange(LONG), at)])
    n = LONG // 2
    first = np.zeros(LONG, dtype=bool)
    first[order[:n]] = True
    for kw, keep in ((dict(), None), (dict(min_p=f(1e-15)), None),
                     (dict(top_k=f(n, torch.int32)), first)):
        token, prob = head.sample_logits(logits, u, **kw)
        for i in range(len(us)):
            check_long_row(row, us[i], int(token[i]), float(prob[i]), keep)
    # top_p of the mass, with u at its end: the nucleus ends with the last token that has a part of it
    w, _ = weights(row)
    c = np.cumsum(w[order].astype(np.longdouble))
    for top_p in (0.99995, 0.99999, 0.7):
        token, prob = head.sample_logits(logits, f(1.0), top_p=f(top_p))
        need = np.longdouble(np.float32(top_p)) * c[-1]
        lo, hi = (int(np.searchsorted(c, need + s * 2.0 ** -35 * c[-1])) for s in (-1, 1))
        last = [int(order[:n + 1].max()) for n in (lo, hi)]
        assert last[0] <= int(token[0]) <= last[1], (top_p, int(token[0]), last)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_sampling_keeps_the_tail_in_rows_of_many(dt):
    """The same where each row is one CTA's and some are left to a second launch."""
    R, V = 160, 1 << 20
    us = np.linspace(0.0, 2.0 ** -17, R, dtype=np.float32)
    logits = torch.full((R, V), -26.5, device="cuda").to(DT[dt])
    logits[:, -1] = 0
    row = f64(logits[0])
    token, prob = head.sample_logits(logits, torch.from_numpy(us).cuda())
    for i in range(0, R, 9):
        check_long_row(row, us[i], int(token[i]), float(prob[i]))


@pytest.mark.parametrize("V", [500, 5003, 65536])
@pytest.mark.parametrize("T", [0.3, 1.0, 1.7])
def test_sampling_next_to_a_border(V, T):
    """u and top_p as near to a border as the definition's answer is still sure, 2^-35 of the mass."""
    R = 24
    g = gen(V)
    logits = 3 * torch.randn(R, V, device="cuda", generator=g)
    ll = f64(logits)
    rng = np.random.default_rng(V)
    cand = (rng.integers(1, 1 << 24, 1 << 20) / 2.0 ** 24).astype(np.float32)
    u, want, near = np.empty(R, np.float32), [], []
    p, last = np.empty(R, np.float32), []
    T32 = float(np.float32(T))

    def closest(c):
        """The candidate whose share of c[-1] is nearest to a border, and its place."""
        c = c.astype(np.float64)  # (summed in more)
        goal = cand.astype(np.float64) * c[-1]
        i = np.searchsorted(c, goal, side="right")
        d = np.minimum(np.abs(goal - np.concatenate([[0], c])[i]), np.abs(c[np.minimum(i, len(c) - 1)] - goal))
        d = np.where(d / c[-1] < 2.0 ** -35, np.inf, d / c[-1])
        b = int(np.argmin(d))
        return cand[b], int(i[b]), float(d[b])

    for r in range(R):
        w, c = weights(ll[r], T32)
        u[r], at, d = closest(c)
        want.append(at)
        near.append(d)
        order = np.argsort(-ll[r], kind="stable")
        p[r], at, _ = closest(np.cumsum(w[order].astype(np.longdouble)))
        last.append(int(order[:at + 1].max()))  # with u = 1: the last of the nucleus
    assert np.median(near) < 2.0 ** -28 or V == 500
    t = torch.full((R,), T, device="cuda")
    token, _ = head.sample_logits(logits, torch.from_numpy(u).cuda(), temperature=t)
    assert token.tolist() == want
    token, _ = head.sample_logits(logits, torch.ones(R, device="cuda"), temperature=t,
                                  top_p=torch.from_numpy(p).cuda())
    assert token.tolist() == last


# ------------------------------------------------------------------------------------- together
def test_first_use_of_a_head_on_another_stream():
    """A call on any stream right after the constructor sees the whole table."""
    V, d, R = 131072, 1024, 16
    g = gen(41)
    w = torch.ones(d, device="cuda").bfloat16()
    x = torch.randn(R, d, device="cuda", generator=g).bfloat16()
    u = torch.rand(R, device="cuda", generator=g)
    side = torch.cuda.Stream()
    for seed in range(4):
        E = torch.randn(V, d, device="cuda", generator=gen(seed)).bfloat16()
        torch.cuda.synchronize()
        hd = head.OutputHead(E, w, out_dtype="fp32")
        first, _ = hd.logits(x, stream=side)
        token, _ = hd.sample(x, u, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(hd.logits(x)[0], first) and torch.equal(hd.sample(x, u)[0], token)


def test_a_head_built_inside_a_capture():
    V, d, R = 3000, 256, 5
    g = gen(42)
    E = torch.randn(V, d, device="cuda", generator=g).bfloat16()
    w = torch.ones(d, device="cuda").bfloat16()
    x = torch.randn(R, d, device="cuda", generator=g).bfloat16()
    want, _ = head.OutputHead(E, w, out_dtype="fp32").logits(x)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out, _ = head.OutputHead(E, w, out_dtype="fp32").logits(x)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_status_calls_beside_products_on_other_streams():
    """Two threads take the error word while products run on their streams."""
    import threading
    ops = operands(300, 5000, 384, 7)
    want = head.matmul_fp8(*ops, out_dtype="fp32")
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(40):
            got = head.matmul_fp8(*ops, out_dtype="fp32", stream=s)
            st = head.head_status(stream=s)  # (synchronises s)
            if st != 0 or not torch.equal(got, want):
                bad.append(st)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


# ------------------------------------------------------------------------------------- long rows
def test_quantising_the_longest_row():
    """2^31 - 1 columns: the last group of eight has seven, and nothing beside them is read or written."""
    n = 2 ** 31 - 1
    x = torch.zeros(n + 9, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(300, device="cuda", generator=gen(3)).bfloat16()
    x[n - 300:n] = tail
    x[n:] = 1e30
    q = torch.full((n + 17,), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((n // 128 + 2,), -1.0, device="cuda")
    args = C.ds_quantize_fp8_args(rows=1, cols=n, dtype=C.DS_DTYPE_BF16, fp8=C.DS_FP8_E4M3, block_rows=1,
                                  x=x.data_ptr(), x_stride=n + 1, q=q.data_ptr(), q_stride=n + 1,
                                  scales=s.data_ptr(), scales_stride=n // 128 + 1)
    C.check(C.load_library().ds_quantize_fp8(ctypes.byref(args), torch.cuda.current_stream().cuda_stream),
            "ds_quantize_fp8")
    torch.cuda.synchronize()
    assert torch.all(q[n:] == 77) and float(s[-1]) == -1.0
    at = n // 128 * 128  # the last block: 127 columns
    y = f64(tail[-(n - at):])[None, :]
    v = quotients(y, "e4m3", 1)
    assert np.array_equal(f64(q[at:n].view(torch.float8_e4m3fn))[None, :], O.fp8_round(v.astype(np.float32), "e4m3"))
    assert abs(float(s[-2]) - np.abs(y).max() / 448) <= 2.0 ** -24 * np.abs(y).max() / 448
    assert int(q[:n - 500].max()) == 0


# ------------------------------------------------------------------------------------- gradients
def test_inputs_that_want_a_gradient():
    """Refused by the operators while gradients are on; constants to a head, as its own weights."""
    g = gen(51)
    E = torch.nn.Parameter(torch.randn(1000, 256, device="cuda", generator=g).bfloat16())
    w = torch.nn.Parameter(torch.ones(256, device="cuda").bfloat16())
    x = torch.randn(3, 256, device="cuda", generator=g).bfloat16()
    u = torch.rand(3, device="cuda", generator=g)
    hd = head.OutputHead(E, w)
    logits, _ = hd.logits(x)
    leaf = x.clone().requires_grad_()
    for call in (lambda: head.rmsnorm_fp8(x, w), lambda: head.rmsnorm_fp8(leaf, w.detach()),
                 lambda: head.rmsnorm_fp8(x, w.detach(), leaf), lambda: head.quantize_fp8(E),
                 lambda: hd.sample(leaf, u), lambda: head.sample_logits(logits.float().requires_grad_(), u)):
        with pytest.raises(ValueError, match="gradient"):
            call()
    with torch.no_grad():
        got, _ = hd.logits(leaf)
        q, _ = head.quantize_fp8(E)
    assert torch.equal(got, logits) and torch.equal(q.view(torch.uint8), hd.q.view(torch.uint8))
    assert not got.requires_grad and not logits.requires_grad


# ------------------------------------------------------------------------------------- special rows
def test_norm_of_each_special_row():
    """With eps = 0: zeros are 0 / 0; squares below fp32's least (|h| below 2^-75) sum to 0, and h / 0
    is infinite; small rows whose squares fp32 holds are rows like others; NaN and infinities."""
    nan, inf = float("nan"), float("inf")
    x = torch.zeros(7, 256, device="cuda")
    x[1, 3] = nan
    x[2] = 1e-30
    x[3] = 1e-18
    x[4, 7], x[4, 200] = inf, 1.0
    x[5, 5] = 1e19
    x[6, 0], x[6, 255] = 2e19, 1.0  # (4e38: the sum overflows)
    w = torch.ones(256, device="cuda")
    q, s, h = head.rmsnorm_fp8(x, w, eps=0.0)
    q, s = f64(q), f64(s)
    tiny = float(np.float32(O.TINY / 448))
    assert h is x
    for r in (0, 1):  # y is NaN throughout, and NaN does not enter a scale
        assert np.isnan(q[r]).all() and (s[r] == tiny).all(), r
    assert np.isnan(q[2]).all() and np.isinf(s[2]).all()
    assert (q[3] == 448).all() and np.allclose(s[3], 1 / 448, rtol=2.0 ** -18, atol=0)
    assert np.isnan(q[4, 7]) and (np.delete(q[4], 7) == 0).all() and (s[4] == tiny).all()
    want = np.zeros(256)
    want[5] = 448
    assert (q[5] == want).all()
    assert np.allclose(s[5], [16 / 448, tiny], rtol=2.0 ** -18, atol=0)
    assert (q[6] == 0).all() and (s[6] == tiny).all()
    q, s, _ = head.rmsnorm_fp8(x[2:3], w, eps=1e-6)  # eps covers it: y = 1e-27, above 2^-100
    assert (f64(q) == 448).all() and np.allclose(f64(s), 1e-27 / 448, rtol=2.0 ** -18, atol=0)


# ------------------------------------------------------------------------------------- no row excused
def away_from_borders(logits, u, kw):
    """u and top_p moved until every row's answer is sure (borders 2^-34 of the mass away): all rows
    can be compared. Returns the expected (token, prob) of each."""
    ll, want = f64(logits), []
    v = {n: t.cpu().numpy() for n, t in kw.items()}
    uu = u.cpu().numpy()
    for r in range(len(ll)):
        for _ in range(30):
            row = {("T" if n == "temperature" else n): t[r].item() for n, t in v.items()}
            token, prob, margin = O.sample_row(ll[r], float(uu[r]), **row)
            if margin >= 2.0 ** -34:
                break
            uu[r] = np.float32((uu[r] + 0.0371) % 1.0)
            if 0 < v["top_p"][r] < 1:
                v["top_p"][r] = np.float32(v["top_p"][r] * 0.9967)
        else:
            raise AssertionError(f"row {r} stays next to a border")
        want.append((token, prob))
    return torch.from_numpy(uu).cuda(), {n: torch.from_numpy(t).cuda() for n, t in v.items()}, want


def rows_of(R, V, seed, kind):
    g = gen(seed)
    if kind == "normal":
        return torch.randn(R, V, device="cuda", generator=g)
    if kind == "steep":
        return 2.0 * -torch.log(torch.rand(R, V, device="cuda", generator=g).clamp(min=1e-9)) - 10
    if kind == "ties":
        return (4 * torch.randn(R, V, device="cuda", generator=g)).round() / 2
    return torch.full((R, V), 0.5, device="cuda")


@pytest.mark.parametrize("R,V", [(400, 5003), (330, 16001), (160, 40009), (24, 262144), (3, 700001)])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_sampling_of_every_row(R, V, dt):
    kinds = [rows_of(-(-R // 4), V, R + i, k) for i, k in enumerate(("normal", "steep", "ties", "flat"))]
    logits = torch.stack(kinds, dim=1).view(-1, V)[:R].contiguous().to(DT[dt])
    pick = lambda *v: torch.tensor([v[(i // 4 + i) % len(v)] for i in range(R)], device="cuda")  # noqa: E731
    kw = dict(temperature=pick(1.0, 0.7, 1.0, 1.3, 0.0, 0.9, 2.0),
              top_k=pick(0, 40, 0, 3000, 0, 0, 1, 0, 0, 0, 700).int(),
              top_p=pick(1.0, 0.9, 0.95, 0.6, 0.9, 1.0, 0.999, 0.8, 0.5),
              min_p=pick(0.0, 0.0, 0.05, 0.0, 0.0, 0.001, 0.0, 0.0))
    u = torch.rand(R, device="cuda", generator=gen(R))
    u, kw, want = away_from_borders(logits, u, kw)
    token, prob = head.sample_logits(logits, u, **kw)
    assert token.tolist() == [t for t, _ in want]
    p = np.array([p for _, p in want])
    assert np.all(np.abs(f64(prob) - p) <= 2.0 ** -20 * p)


# ------------------------------------------------------------------------------------- captures
def test_the_first_calls_of_a_process_inside_a_capture():
    """What the library sets up once a device may be set up while a stream is being captured."""
    import os
    import subprocess
    import sys
    code = """
import torch
from canvas_sampler_gb300 import head
g = torch.Generator(device="cuda"); g.manual_seed(1)
x = torch.randn(400, 512, device="cuda", generator=g).bfloat16()
E = torch.randn(6000, 512, device="cuda", generator=g).bfloat16()
w = torch.ones(512, device="cuda").bfloat16()
u = torch.rand(400, device="cuda", generator=g)
p = torch.full((400,), 0.97, device="cuda")
def run():
    q, s = head.quantize_fp8(E)
    a, sa, _ = head.rmsnorm_fp8(x, w)
    y = head.matmul_fp8(a, sa, q, s, out_dtype="fp32")
    few = head.matmul_fp8(a[:3], sa[:3], q, s)
    return y, few, *head.sample_logits(y, u, top_p=p), *head.sample_logits(few, u[:3], top_p=p[:3])
torch.cuda.synchronize()
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    out = run()
gr.replay()
torch.cuda.synchronize()
got = [t.clone() for t in out]
want = run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert head.head_status() == 0
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_two_graphs_replayed_at_once():
    """Two captured calls on two streams share nothing but the weights."""
    g = gen(61)
    E = torch.randn(20000, 256, device="cuda", generator=g).bfloat16()
    hd = head.OutputHead(E, torch.ones(256, device="cuda").bfloat16())
    R = 400
    sets = [torch.randn(R, 256, device="cuda", generator=g).bfloat16() for _ in range(2)]
    u = torch.rand(R, device="cuda", generator=g)
    kw = dict(top_p=torch.full((R,), 0.97, device="cuda"),
              top_k=(torch.arange(R, device="cuda") % 3 * 1000).int())
    want = [hd.sample(x, u, **kw) for x in sets]
    torch.cuda.synchronize()
    graphs = []
    for x in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = hd.sample(x, u, **kw)
        graphs.append((gr, out, torch.cuda.Stream()))
    for _ in range(10):
        for _, out, _ in graphs:
            out[0].fill_(-5)
        torch.cuda.synchronize()
        for gr, _, s in graphs:
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for (_, out, _), w in zip(graphs, want):
            assert torch.equal(out[0], w[0]) and torch.equal(out[1], w[1])

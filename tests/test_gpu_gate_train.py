"""The calls that train the gate against the fp64 oracle.

Tolerances follow from the arithmetic.  u = 2^-24 is half a step of fp32; a
sum of n fp32 terms in any order is off by at most gamma_n = n u / (1 - n u)
of the sum of their magnitudes.  Probabilities: exp is ex2.approx (2 ulp, 4 u) of
the rounded difference D = max - logit times log2 e; the difference is off by D u,
the product by D u again and log2 e as a float by 0.22 D u, so exp by (2.22 D + 4) u,
its numerators and their sum by as much: a softmax over E values is off by
(4.44 D + E + 16) u relative (numerator, sum, sum's adds, reciprocal, product).  bf16 results round once more, by 2^-8 of the value
at most."""

import math

import numpy as np
import pytest
import torch

import routing_dispatch_expert_softmax_b200 as moe
from oracle import gate_train_oracle as go
from routing_dispatch_expert_softmax_b200.binding import MoEShape

from parity_utils import U32, np64

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.load_library()
    yield
    torch.cuda.synchronize()


def dev(a, dtype=None):
    return torch.as_tensor(a, dtype=dtype).to(DEV)


def clean(ws):
    st = moe.moe_check(ws)
    assert st == moe.MOE_OK, moe.moe_error_string(st)


def within(got, ref, bound, what):
    got, ref = np64(got), np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    off = np.abs(got - ref)
    assert np.all(off <= bound), (what, float(np.max(off - bound)), float(np.max(off)))


# ---------------------------------------------------------------- gate batch
class Batch:
    """Logits, selections and gates of T tokens, with sequences and a mask."""

    def __init__(self, T, E, k, seqs=None, masked=False, seed=0, scale=1.5):
        r = np.random.default_rng(seed)
        self.T, self.E, self.k = T, E, k
        self.L = (r.normal(size=(T, E)) * scale - 0.3 * np.log(r.permutation(E) + 1)).astype(np.float32)
        self.idx = np.argsort(-self.L, axis=1, kind="stable")[:, :k].astype(np.int32)
        top = np.take_along_axis(self.L, self.idx, 1).astype(np.float64)
        w = np.exp(top - top[:, :1])
        self.w = (w / w.sum(1, keepdims=True)).astype(np.float32)
        self.dw = r.normal(size=(T, k)).astype(np.float32)
        self.mask = (r.random(T) > 0.2).astype(np.uint8) if masked else None
        self.seqs = seqs
        self.S = 1 if seqs is None else len(seqs) - 1
        self.shape = MoEShape.of(T, 64, E, k, 64)
        self.a, self.b, self.g = 0.02, 0.003, 0.75

    def device(self):
        self.ws = moe.workspace_bwd(self.shape, self.S)
        self.dL, self.didx = dev(self.L), dev(self.idx)
        self.dw_, self.w_ = dev(self.dw), dev(self.w)
        self.dg = dev([self.g], torch.float32)
        self.dmask = None if self.mask is None else dev(self.mask)
        self.dseqs = None if self.seqs is None else dev(np.asarray(self.seqs, dtype=np.int32))
        # poisoned outputs: what a call leaves unwritten shows
        self.loss = torch.full((3,), math.nan, device=DEV)
        self.counts = torch.full((self.S, self.E), -7, dtype=torch.int32, device=DEV)
        self.tokens = torch.full((self.S + 2,), -7, dtype=torch.int32, device=DEV)
        self.mean = torch.full((self.S, self.E), math.nan, device=DEV)
        self.dlogits = torch.full((self.T, self.E), math.nan, device=DEV)
        return self

    def run_loss(self, **kw):
        moe.moe_balance_loss(self.dL, self.didx, self.loss, self.counts, self.tokens, self.shape,
                             self.ws, **dict(dict(balance_coef=self.a, z_coef=self.b,
                                                  token_mask=self.dmask, seq_offsets=self.dseqs,
                                                  prob_mean=self.mean), **kw))

    def run_bwd(self, gates=True, aux=True, **kw):
        moe.moe_gate_bwd(self.dL if aux else None, self.didx if gates else None, self.dlogits,
                         self.shape, self.ws,
                         **dict(dict(w=self.w_ if gates else None, dw=self.dw_ if gates else None,
                                     counts=self.counts if aux else None,
                                     tokens=self.tokens if aux else None, balance_coef=self.a,
                                     z_coef=self.b, dloss=self.dg,
                                     token_mask=self.dmask, seq_offsets=self.dseqs), **kw))


def softmax_rel(b):
    """Relative error bound of each row's probabilities."""
    L = np.where(np.isfinite(b.L), b.L, np.nan).astype(np.float64)
    with np.errstate(all="ignore"):
        D = np.nan_to_num(np.nanmax(L, 1) - np.nanmin(L, 1))
    return (4.44 * D + b.E + 16) * U32


def check_loss(b):
    loss, counts, tokens, mean = go.balance_loss(b.L, b.idx, b.a, b.b, b.mask, b.seqs)
    assert np.array_equal(b.counts.cpu().numpy(), counts)
    assert np.array_equal(b.tokens.cpu().numpy(), tokens)
    # a block sums at most ceil(T / 296) + 32 rows in fp32, warps' sums 8 more; then fp64
    n = -(-b.T // 296) + 32 + 8
    rel = float(softmax_rel(b).max()) + (n + 4) * U32
    within(b.mean, mean, rel * mean + 1e-37, "prob_mean")
    with np.errstate(all="ignore"):
        lse = np.array([go.softmax_lse(r)[1] for r in b.L.astype(np.float64)])
    lse = lse[np.isfinite(lse)]
    # __logf of a sum in [1, E]: 2^-21.41 up to 2, 3 ulp (6 u) of at most log E above; the
    # sum's own error, the two adds
    d = U32 * (2 * np.abs(lse) + 6.1 + 6 * math.log(max(2, b.E))) + float(softmax_rel(b).max())
    zb = b.b * (float(np.max(2 * np.abs(lse) * d + d * d, initial=0)) + (n + 4) * U32 * float(np.max(lse ** 2, initial=0)))
    got = np64(b.loss)
    lb = (rel + 4 * U32) * abs(loss[1])
    assert abs(got[1] - loss[1]) <= lb, (got, loss)
    assert abs(got[2] - loss[2]) <= zb + 2 * U32 * abs(loss[2]), (got, loss)
    assert abs(got[0] - loss[0]) <= lb + zb + 2 * U32 * abs(loss[0]), (got, loss)


def check_bwd(b, gates=True, aux=True):
    counts = b.counts.cpu().numpy() if aux else None
    ref = go.gate_bwd(b.L, b.idx, np64(b.w_), np64(b.dw_) if gates else None, counts, b.a, b.b,
                      b.g, b.mask, b.seqs)
    bound = np.zeros_like(ref)
    if aux:
        rel = softmax_rel(b)
        rows = go._rows(b.T, b.mask, b.seqs, b.L.astype(np.float64))
        live, total = max(1, sum(len(r) > 0 for r in rows)), max(1, sum(len(r) for r in rows))
        for i, r in enumerate(rows):
            for t in r:
                p, lse = go.softmax_lse(b.L[t].astype(np.float64))
                f = b.g * b.a * b.E / (live * b.k * len(r) ** 2) * counts[i]
                dot, z = float(f @ p), abs(2 * b.b * b.g / total * lse)
                dl = U32 * (2 * abs(lse) + 6.1 + 6 * math.log(max(2, b.E))) + rel[t]
                # f: 8 roundings; dot: a sum of E products of p and f; z: lse's error and 4 roundings
                bound[t] = p * ((rel[t] + 12 * U32) * (f + dot + z)
                                + (rel[t] + (b.E + 12) * U32) * dot
                                + 2 * b.b * b.g / total * dl + 6 * U32 * z) + 1e-37
    if gates:
        for t in range(b.T):
            s = float(np.abs(b.w[t].astype(np.float64) * b.dw[t]).sum())
            for j, e in enumerate(b.idx[t]):
                bound[t, e] += U32 * ((b.k + 6) * s * b.w[t, j] + 4 * abs(b.w[t, j] * b.dw[t, j]))
    within(b.dlogits, ref, bound + 2 * U32 * np.abs(ref), "dlogits")


SIZES = [(1, 1, 1), (1, 2, 1), (3, 4, 4), (64, 8, 2), (33, 5, 3), (17, 13, 13), (31, 24, 7),
         (5, 33, 8), (40, 64, 6), (257, 100, 8), (129, 128, 8), (70, 130, 9), (61, 256, 8),
         (37, 300, 32), (20, 512, 5), (11, 1000, 32), (9, 1024, 8), (1000, 6, 2), (2000, 33, 4),
         (1030, 256, 8), (300, 700, 3)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("masked", [False, True])
def test_loss_and_gradient(T, E, k, masked):
    b = Batch(T, E, k, masked=masked, seed=T + E).device()
    b.run_loss()
    clean(b.ws)
    check_loss(b)
    b.run_bwd()
    clean(b.ws)
    check_bwd(b)


@pytest.mark.parametrize("T,E,k,seqs", [
    (100, 8, 2, [0, 100]), (100, 8, 2, [0, 1, 1, 2, 50, 99]), (100, 16, 4, [7, 20, 64, 64, 90]),
    (64, 64, 8, list(range(65))), (300, 128, 8, [0, 0, 31, 32, 33, 200, 300, 300]),
    (200, 256, 8, [200, 200]), (200, 40, 3, [0, 0, 0]), (129, 300, 4, [5, 6, 128])])
@pytest.mark.parametrize("masked", [False, True])
def test_sequences(T, E, k, seqs, masked):
    b = Batch(T, E, k, seqs=seqs, masked=masked, seed=T).device()
    b.run_loss()
    clean(b.ws)
    check_loss(b)
    b.run_bwd()
    clean(b.ws)
    check_bwd(b)


@pytest.mark.parametrize("T,E,k,S", [(20000, 16, 2, 1), (20000, 16, 2, 700), (19000, 128, 4, 1)])
def test_many_tokens(T, E, k, S):
    # more tokens than 32 for each of 592 blocks: longer blocks
    r = np.random.default_rng(1)
    seqs = None if S == 1 else np.concatenate([[0], np.sort(r.integers(0, T, S - 1)), [T - 5]])
    b = Batch(T, E, k, seqs=seqs, masked=True, seed=2).device()
    b.run_loss()
    b.run_bwd()
    clean(b.ws)
    check_loss(b)
    check_bwd(b)


@pytest.mark.parametrize("gates,aux", [(True, False), (False, True)])
@pytest.mark.parametrize("E", [8, 48, 260])
def test_one_part_alone(gates, aux, E):
    b = Batch(50, E, 3, seed=E).device()
    b.run_loss()
    b.run_bwd(gates=gates, aux=aux)
    check_bwd(b, gates=gates, aux=aux)
    clean(b.ws)


def test_coefficients_of_zero_leave_terms_out():
    b = Batch(40, 8, 2, seed=5)
    b.L[3] = np.finfo(np.float32).min  # lse^2 overflows: 0 times it may not show
    b.b = 0.0
    b.device()
    b.run_loss()
    b.run_bwd()
    check_loss(b)
    check_bwd(b)
    assert b.loss[2].item() == 0.0


def test_rows_of_the_lowest_value_and_masked_experts():
    b = Batch(64, 48, 4, seed=6)
    b.L[5, 10:] = -np.inf                       # experts that are masked out
    b.L[6] = -np.inf                            # nothing is left: the token does not count
    b.L[7, 1:] = np.finfo(np.float32).min       # one expert far above the others
    b.L[8] = -1e30                              # uniform, far from zero
    b.b = 1e-38                                 # keeps lse^2 of that row finite
    b.device()
    b.run_loss()
    clean(b.ws)
    assert b.tokens.cpu().tolist() == [63, 63, 1]
    loss, counts, _, mean = go.balance_loss(b.L, b.idx, b.a, 0.0)
    assert np.array_equal(b.counts.cpu().numpy(), counts)
    rel = (4.44 * 12 + b.E + 60) * U32
    within(b.mean, mean, rel * mean + 1e-37, "prob_mean")
    assert abs(b.loss[1].item() - loss[1]) <= (rel + 4 * U32) * loss[1]
    b.run_bwd()
    out = np64(b.dlogits)
    assert np.all(np.isfinite(out))
    alone = np.zeros_like(out[6])
    dot = float(b.w[6].astype(np.float64) @ b.dw[6])
    alone[b.idx[6]] = b.w[6] * (b.dw[6] - dot)
    assert np.allclose(out[6], alone, rtol=0, atol=16 * U32)  # the gates' part alone


def test_uncounted_values_do_not_leak():
    T, E, k = 90, 24, 3
    b = Batch(T, E, k, seqs=[10, 40, 80], masked=True, seed=8)
    plain = Batch(T, E, k, seqs=[10, 40, 80], masked=True, seed=8).device()
    out = [t for t in range(T) if t < 10 or t >= 80 or not b.mask[t]]
    b.L[out] = np.nan
    b.L[out[::2]] = np.inf
    b.device()
    for q in (plain, b):
        q.run_loss()
        q.run_bwd()
        clean(q.ws)
    for name in ("loss", "counts", "tokens", "mean", "dlogits"):
        assert torch.equal(getattr(b, name), getattr(plain, name)), name


def test_nan_and_inf_show():
    for bad in (np.nan, np.inf):
        b = Batch(50, 8, 2, seqs=[0, 20, 50], seed=9)
        b.L[30, 3] = bad
        b.device()
        b.run_loss()
        assert torch.isnan(b.loss[:2]).all()
        assert torch.isfinite(b.mean[0]).all() and torch.isnan(b.mean[1]).any()


def test_nothing_counts():
    for kw in (dict(mask=True), dict(seqs=[30, 30])):
        b = Batch(30, 8, 2, seqs=kw.get("seqs"), seed=1)
        if "mask" in kw:
            b.mask = np.zeros(30, dtype=np.uint8)
        b.device()
        b.run_loss()
        b.run_bwd(gates=False)
        assert b.loss.tolist() == [0, 0, 0] and not b.counts.any() and not b.tokens.any()
        assert not b.mean.any() and not b.dlogits.any()
    e = Batch(0, 8, 2, seqs=[0, 0, 0]).device()
    e.run_loss()
    assert e.loss.tolist() == [0, 0, 0] and not e.counts.any() and not e.tokens.any()


def test_bad_offsets_and_ids_are_recorded():
    for seqs in ([0, 30, 20, 50], [-1, 50], [0, 51]):
        b = Batch(50, 8, 2, seqs=seqs, seed=3).device()
        b.run_loss()
        assert moe.moe_check(b.ws) == moe.MOE_ERR_DEVICE_CHECK
    b = Batch(50, 8, 2, seed=3)
    b.idx[7, 1], b.idx[9, 0] = 8, -1
    b.device()
    b.run_loss()
    assert moe.moe_check(b.ws) == moe.MOE_ERR_DEVICE_CHECK
    assert int(b.counts.sum()) == 98 and b.tokens.tolist() == [50, 50, 1]
    b.run_bwd()
    assert moe.moe_check(b.ws) == moe.MOE_ERR_DEVICE_CHECK
    assert moe.moe_check(b.ws) == moe.MOE_OK
    assert torch.isfinite(b.dlogits).all()


@pytest.mark.parametrize("E,k", [(8, 8), (8, 3), (64, 12), (200, 32)])
def test_one_expert_named_twice(E, k):
    b = Batch(30, E, k, seed=4)
    b.idx[:, 1] = b.idx[:, 0]
    b.idx[5] = b.idx[5, 0]
    b.device()
    b.run_loss()
    b.run_bwd()
    check_loss(b)
    first = b.dlogits.clone()
    check_bwd(b)
    for _ in range(3):
        b.run_bwd()
        assert torch.equal(first, b.dlogits)


def test_same_bits_every_time():
    b = Batch(5000, 128, 8, seqs=[0, 100, 100, 4000, 4990], masked=True, seed=11).device()
    b.run_loss()
    want = [b.loss.clone(), b.mean.clone()]
    for _ in range(5):
        b.run_loss()
        assert torch.equal(b.loss, want[0]) and torch.equal(b.mean, want[1])


def test_offset_views():
    # 4-byte aligned bases: the 16-byte path may not be taken
    b = Batch(40, 16, 2, seed=12).device()
    big = torch.zeros(40 * 16 + 1, device=DEV)
    out = torch.full((40 * 16 + 3,), math.nan, device=DEV)
    big[1:] = b.dL.view(-1)
    b.dL, b.dlogits = big[1:].view(40, 16), out[1:-2].view(40, 16)
    b.run_loss()
    b.run_bwd()
    check_loss(b)
    check_bwd(b)
    assert torch.isnan(out[0]) and torch.isnan(out[-2:]).all()


# ------------------------------------------------------------------- combine
@pytest.mark.parametrize("T,d,k", [(1, 64, 1), (1, 7168, 8), (3, 128, 5), (64, 2048, 8), (37, 320, 3),
                                   (700, 192, 4), (2500, 64, 2), (300, 1024, 32)])
@pytest.mark.parametrize("want", ["both", "dw", "dz"])
def test_combine_bwd(T, d, k, want):
    g = torch.Generator(device=DEV).manual_seed(T * k + d)
    dy = torch.randn(T, d, generator=g, device=DEV).bfloat16()
    z = torch.randn(T * k, d, generator=g, device=DEV).bfloat16()
    row = torch.randperm(T * k, generator=g, device=DEV).int().view(T, k)
    w = torch.rand(T, k, generator=g, device=DEV)
    s = MoEShape.of(T, d, k, k, 64)
    dw = torch.full((T, k), math.nan, device=DEV) if want != "dz" else None
    dz = torch.full((T * k, d), math.nan, dtype=torch.bfloat16, device=DEV) if want != "dw" else None
    moe.moe_combine_bwd(dy, z if dw is not None else None, row, w if dz is not None else None, s,
                        dw=dw, dz=dz)
    rdw, rdz = go.combine_bwd(np64(dy), np64(z), row.cpu().numpy(), np64(w))
    if dw is not None:
        mags = np.abs(np64(dy))[:, None, :] * np.abs(np64(z)[row.cpu().numpy().reshape(-1)]).reshape(T, k, d)
        n = d + 8
        within(dw, rdw, n * U32 / (1 - n * U32) * mags.sum(2), "dw")
    if dz is not None:
        within(dz, rdz, (BF16 * (1 + U32) + 2 * U32) * np.abs(rdz), "dz")


def test_combine_bwd_bad_rows_and_untouched_rows():
    T, d, k = 20, 128, 2
    s = MoEShape.of(T, d, 2, k, 64)
    dy, z = torch.ones(T, d, device=DEV).bfloat16(), torch.ones(T * k, d, device=DEV).bfloat16()
    row = torch.arange(T * k, device=DEV).int().view(T, k)
    row[3, 1], row[4, 0] = T * k, -1
    dw = torch.full((T, k), math.nan, device=DEV)
    dz = torch.full((T * k, d), 7.0, device=DEV).bfloat16()
    moe.moe_combine_bwd(dy, z, row, torch.ones(T, k, device=DEV), s, dw=dw, dz=dz)
    want = torch.full((T, k), float(d), device=DEV)
    want[3, 1] = want[4, 0] = 0
    assert torch.equal(dw, want)
    left = torch.ones(T * k, d, device=DEV).bfloat16()
    left[7] = left[8] = 7.0
    assert torch.equal(dz, left)


# -------------------------------------------------------------------- router
def check_router(T, d, E, dw=True, db=True, dx=True, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed + T + d + E)
    x = torch.randn(T, d, generator=g, device=DEV).bfloat16()
    W = torch.randn(d, E, generator=g, device=DEV) / math.sqrt(d)
    dl = torch.randn(T, E, generator=g, device=DEV) * torch.rand(T, 1, generator=g, device=DEV) * scale
    s = MoEShape.of(T, d, E, 1, 64)
    ws = moe.workspace_bwd(s)
    ws[256:] = 0xff  # NaN patterns: scratch that is read before it is written shows
    out = dict(dw_g=torch.full((d, E), math.nan, device=DEV) if dw else None,
               dbias=torch.full((E,), math.nan, device=DEV) if db else None,
               dx=torch.full((T, d), math.nan, dtype=torch.bfloat16, device=DEV) if dx else None)
    moe.moe_router_bwd(x if dw else None, W if dx else None, dl, s, ws, **out)
    clean(ws)
    # the 64-bit products on the device (the same formula as the oracle's)
    x64, W64, l64 = x.double(), W.double(), dl.double()
    if dw:
        # three products a term, fp32 sums that may truncate (unit 2u)
        n = 3 * T + 16
        bound = n * 2 * U32 / (1 - n * 2 * U32) * (x64.abs().t() @ l64.abs())
        off = (out["dw_g"].double() - x64.t() @ l64).abs()
        assert bool((off <= bound + 1e-37).all()), ("dw_g", float((off - bound).max()))
    if db:
        bound = (T + 4) * U32 / (1 - (T + 4) * U32) * l64.abs().sum(0)
        off = (out["dbias"].double() - l64.sum(0)).abs()
        assert bool((off <= bound + 1e-37).all()), ("dbias", float((off - bound).max()))
    if dx:
        ref = l64 @ W64.t()
        # Both operands are rounded to fp16 after a power of two brings their row's
        # largest value to [2^14, 2^15): off by 2^-11 of the value while that is
        # normal (2^-14 up), else by half of 2^-24, which is 2^-39 of the row's largest.
        # A product is then off by 2^-10 + 2^-22 and the rows' 2^-39 terms.  Sums in
        # fp32 that may truncate, two scalings back.
        n = E + 16
        mags = l64.abs() @ W64.abs().t()
        low = 2.0 ** -39 * (l64.abs().amax(1)[:, None] * W64.abs().sum(1)[None, :]
                            + l64.abs().sum(1)[:, None] * W64.abs().amax(1)[None, :])
        bound = BF16 * ref.abs() + (1 + BF16) * ((2.0 ** -10 + 2.0 ** -22 + n * 2 * U32) * mags
                                                 + 1.01 * low)
        off = (out["dx"].double() - ref).abs()
        assert bool((off <= bound + 1e-37).all()), ("dx", float((off - bound).max()))
    return x, W, dl, s, ws, out


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 127, 129, 300])
@pytest.mark.parametrize("d,E", [(64, 1), (64, 8), (128, 65), (192, 128), (256, 130), (320, 256)])
def test_router_bwd(T, d, E):
    check_router(T, d, E)


@pytest.mark.parametrize("T,d,E", [(64, 2048, 128), (1000, 2048, 128), (257, 7168, 256), (33, 64, 1024),
                                   (515, 128, 1000), (20000, 64, 8), (4097, 448, 60), (700, 16384, 4)])
def test_router_bwd_larger(T, d, E):
    check_router(T, d, E)


@pytest.mark.parametrize("which", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1)])
def test_router_bwd_parts(which):
    check_router(150, 192, 24, *map(bool, which))


def test_router_bwd_tiny_and_huge_gradients():
    check_router(100, 64, 16, scale=1e-30)
    check_router(300, 192, 40, scale=3e-34)
    check_router(100, 64, 16, scale=1e30)


@pytest.mark.parametrize("T", [1, 7, 15, 16, 17, 32, 33, 63, 64, 65, 96, 97, 128, 129, 192, 193])
@pytest.mark.parametrize("d,E", [(64, 1), (64, 3), (128, 8), (448, 60), (1088, 130), (4672, 36), (4736, 9), (4800, 16),
                                 (64, 255), (128, 260), (64, 640), (9472, 5), (9536, 5), (2368, 8), (2432, 8)])
def test_router_bwd_few_tokens(T, d, E):
    check_router(T, d, E)


@pytest.mark.parametrize("which", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1)])
@pytest.mark.parametrize("T", [5, 50, 90, 110, 190])
def test_router_bwd_few_tokens_parts(T, which):
    check_router(T, 192, 24, *map(bool, which))


@pytest.mark.parametrize("scale", [1e-30, 3e-34, 1e30])
def test_router_bwd_few_tokens_tiny_and_huge_gradients(scale):
    check_router(40, 128, 20, scale=scale)
    check_router(180, 64, 12, scale=scale)


def test_router_bwd_few_tokens_same_bits_and_unaligned():
    x, W, dl, s, ws, out = check_router(37, 256, 12)
    want = {n: t.clone() for n, t in out.items()}
    # dlogits and the fp32 outputs may start on any element
    dl1 = torch.empty(dl.numel() + 1, device=DEV)[1:].view_as(dl).copy_(dl)
    W1 = torch.empty(W.numel() + 1, device=DEV)[1:].view_as(W).copy_(W)
    buf = torch.full((out["dw_g"].numel() + 2,), 7.0, device=DEV)
    out1 = dict(out, dw_g=buf[1:-1].view_as(W))
    for _ in range(3):
        moe.moe_router_bwd(x, W1, dl1, s, ws, **out1)
        assert all(torch.equal(want[n], out1[n]) for n in want)
    assert buf[0] == 7 and buf[-1] == 7


def test_router_bwd_few_tokens_infinite_gradient_shows():
    x, W, dl, s, ws, out = check_router(20, 64, 8)
    dl[3, 2] = math.inf
    dl[5, 4] = math.nan
    moe.moe_router_bwd(x, W, dl, s, ws, **out)
    for e in (2, 4):
        assert not torch.isfinite(out["dw_g"][:, e]).any() and not torch.isfinite(out["dbias"][e])
    good = [0, 1, 3, 5, 6, 7]
    assert torch.isfinite(out["dw_g"][:, good]).all() and torch.isfinite(out["dbias"][good]).all()
    assert not torch.isfinite(out["dx"][[3, 5]]).any()
    assert torch.isfinite(out["dx"][[0, 1, 2, 4, 19]]).all()


def test_router_bwd_no_tokens():
    s = MoEShape.of(0, 128, 8, 1, 64)
    ws = moe.workspace_bwd(s)
    dw, db = torch.ones(128, 8, device=DEV), torch.ones(8, device=DEV)
    moe.moe_router_bwd(torch.empty(0, 128, device=DEV).bfloat16(), torch.ones(128, 8, device=DEV),
                       torch.empty(0, 8, device=DEV), s, ws, dw_g=dw, dbias=db,
                       dx=torch.empty(0, 128, device=DEV).bfloat16())
    assert not dw.any() and not db.any()


def test_router_bwd_same_bits_every_time():
    x, W, dl, s, ws, out = check_router(3000, 256, 40)
    want = {n: t.clone() for n, t in out.items()}
    for _ in range(4):
        moe.moe_router_bwd(x, W, dl, s, ws, **out)
        assert all(torch.equal(want[n], out[n]) for n in want)


def test_router_bwd_infinite_gradient_shows():
    x, W, dl, s, ws, out = check_router(70, 64, 8)
    dl[3, 2] = math.inf
    dl[5, 4] = math.nan
    moe.moe_router_bwd(x, W, dl, s, ws, **out)
    for e in (2, 4):
        assert not torch.isfinite(out["dw_g"][:, e]).any() and not torch.isfinite(out["dbias"][e])
    good = [0, 1, 3, 5, 6, 7]
    assert torch.isfinite(out["dw_g"][:, good]).all() and torch.isfinite(out["dbias"][good]).all()
    assert not torch.isfinite(out["dx"][[3, 5]]).any()
    assert torch.isfinite(out["dx"][[0, 1, 2, 4, 69]]).all()


# ---------------------------------------------------------------------- clip
def check_clip(sizes, dtypes, max_norm, out_dtypes=None, scale=1.0, offset=0):
    """In place (out_dtypes None) or into separate tensors; every tensor is a
    slice of a larger one, `offset` elements in, whose margins must survive."""
    r = np.random.default_rng(len(sizes) + sum(sizes) % 1000)
    bufs, grads = [], []
    for n, t in zip(sizes, dtypes):
        buf = dev((r.normal(size=n + offset + 3) * scale).astype(np.float32)).to(t)
        bufs.append(buf)
        grads.append(buf[offset:offset + n])
    before = [b.clone() for b in bufs]
    ref_norm, ref = go.clip_grads([np64(g) for g in grads], max_norm)
    outs = None
    if out_dtypes is not None:
        outs = [torch.full((n,), math.nan, dtype=t, device=DEV) for n, t in zip(sizes, out_dtypes)]
    norm = torch.full((1,), math.nan, device=DEV)
    lst = moe.GradList(grads, outs)
    moe.moe_clip_grads(lst, max_norm, norm)
    clean(lst.ws)
    # sums of at most 8 squares in fp32 (8 u of them, 4 u of the norm), theirs in fp64
    # (off by n 2^-53), one rounding of the norm
    assert abs(norm.item() - ref_norm) <= (5.1 * U32 + sum(sizes) * 2.0 ** -53) * ref_norm
    for got, want in zip(grads if outs is None else outs, ref):
        half = BF16 if got.dtype == torch.bfloat16 else U32
        # the factor's norm (5 u), the factor and the product rounded to fp32, then the
        # result's own rounding
        within(got, want, (half + 8 * U32) * np.abs(want) + (1e-40 if scale < 1e-20 else 0), "out")
    for b, old, n in zip(bufs, before, sizes):
        assert torch.equal(b[:offset], old[:offset]) and torch.equal(b[offset + n:], old[offset + n:])
        if outs is not None:
            assert torch.equal(b, old)


F, H = torch.float32, torch.bfloat16


@pytest.mark.parametrize("max_norm", [0.5, 1e6, math.inf, 0.0])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_clip_in_place(max_norm, offset):
    check_clip([5, 1, 4096, 2049, 70000], [F, H, H, F, H], max_norm, offset=offset)


@pytest.mark.parametrize("max_norm", [0.5, math.inf])
@pytest.mark.parametrize("offset", [0, 2, 5])
def test_clip_into_other_tensors(max_norm, offset):
    check_clip([7, 300, 9001, 33333, 64], [F, H, H, F, H], max_norm, [F, F, H, F, H], offset=offset)


@pytest.mark.parametrize("max_norm", [0.5, math.inf])
@pytest.mark.parametrize("types", [(F, F), (H, H), (H, F)])
def test_clip_into_a_flat_buffer(max_norm, types):
    # every alignment of a gradient against its slice of the buffer
    sizes = [1, 2, 3, 5, 7, 8, 9, 15, 16, 17, 31, 63, 2047, 2049, 4097, 33, 6145, 12289]
    r = np.random.default_rng(1)
    for shift in range(8):
        big = [dev(r.normal(size=n + shift).astype(np.float32)).to(types[0]) for n in sizes]
        grads = [b[shift:] for b in big]
        flat = torch.full((sum(sizes) + 1,), math.nan, dtype=types[1], device=DEV)
        outs, at = [], 0
        for n in sizes:
            outs.append(flat[at:at + n])
            at += n
        _, ref = go.clip_grads([np64(g) for g in grads], max_norm)
        moe.moe_clip_grads(moe.GradList(grads, outs), max_norm)
        half = BF16 if types[1] == H else U32
        for o, w in zip(outs, ref):
            within(o, w, (half + 8 * U32) * np.abs(w), "out")
        assert torch.isnan(flat[-1])


@pytest.mark.parametrize("n", [1, 64, 65, 767, 768, 769, 1600])
def test_clip_many_tensors(n):
    r = np.random.default_rng(n)
    check_clip([int(v) for v in r.integers(0, 300, n)], [H if i % 3 else F for i in range(n)], 1.0)


def test_clip_large_and_uneven():
    check_clip([3_000_001, 1, 1_500_000], [H, F, F], 2.0)


def test_clip_extreme_values():
    check_clip([1000, 1000], [F, F], 1.0, scale=1e30)      # squares pass the fp32 range
    check_clip([1000, 1000], [F, H], 1e-32, scale=1e-28)   # ... or vanish in it
    check_clip([1000, 1000], [F, H], 1e-12, scale=1e-15)   # ... or come near its lowest


def test_clip_mostly_zeros():
    g = torch.zeros(100000, device=DEV)
    g[::977] = torch.arange(1, 104, device=DEV, dtype=torch.float32) * 1e-3
    ref, want = go.clip_grads([np64(g)], 0.1)
    norm = torch.empty(1, device=DEV)
    moe.moe_clip_grads([g], 0.1, norm)
    assert abs(norm.item() - ref) <= 5.1 * U32 * ref
    within(g, want[0], 9 * U32 * np.abs(want[0]), "scaled")


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_clip_not_finite_leaves_gradients(bad):
    g = [torch.randn(100, device=DEV), torch.randn(50, device=DEV).bfloat16()]
    g[1][7] = bad
    want = [t.clone() for t in g]
    out = [torch.empty_like(t) for t in g]
    norm = torch.zeros(1, device=DEV)
    moe.moe_clip_grads(g, 1.0, norm)
    assert not math.isfinite(norm.item())
    moe.moe_clip_grads(moe.GradList(g, out), 1.0)
    for a, b, c in zip(g, want, out):
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
        assert torch.equal(torch.nan_to_num(c), torch.nan_to_num(b))


def test_clip_two_halves_add_up():
    # the norm over two ranks' gradients: each sums its own, the sums are added
    a, b = [torch.randn(5000, device=DEV)], [torch.randn(7000, device=DEV).bfloat16()]
    ref, want = go.clip_grads([np64(a[0]), np64(b[0])], 3.0)
    sums = torch.full((2,), math.nan, dtype=torch.float64, device=DEV)
    moe.moe_grad_sumsq(a, sums[:1])
    moe.moe_grad_sumsq(b, sums[1:])
    total, norm = sums.sum().view(1), torch.empty(1, device=DEV)
    for g, w in ((a, want[0]), (b, want[1])):
        moe.moe_grad_scale(g, total, 3.0, norm)
        assert abs(norm.item() - ref) <= 5.1 * U32 * ref
        within(g[0], w, (BF16 if g[0].dtype == H else U32) * np.abs(w) + 8 * U32 * np.abs(w), "scaled")


def test_clip_list_follows_moved_tensors():
    p = torch.randn(64, device=DEV)
    lst = moe.GradList([p])
    norm = torch.empty(1, device=DEV)
    moe.moe_clip_grads(lst, math.inf, norm)
    p.data = torch.full((64,), 2.0, device=DEV)
    moe.moe_clip_grads(lst, 1.0, norm)
    assert norm.item() == 16.0
    assert torch.allclose(p, torch.full_like(p, 2.0 / (16 + 1e-6)), rtol=1e-6)


def test_clip_refuses_shared_memory():
    buf, other = torch.zeros(100, device=DEV), torch.zeros(100, device=DEV)
    a, b = buf[:50], buf[40:]
    with pytest.raises(ValueError, match="overlaps"):
        moe.GradList([a, b])                       # both scaled in place
    with pytest.raises(ValueError, match="overlaps"):
        moe.GradList([a, a])
    with pytest.raises(ValueError, match="overlaps"):
        moe.GradList([a], [buf[10:60]])
    with pytest.raises(ValueError, match="overlaps"):
        moe.GradList([a, other[:50]], [buf[45:95], other[50:]])
    with pytest.raises(ValueError, match="overlaps"):
        moe.GradList([a, other[:60]], [other[10:60], buf[40:]])
    moe.GradList([a, b], [other[:50], torch.zeros(60, device=DEV)])  # read twice only
    moe.GradList([a, buf[50:]])


def test_clip_nothing():
    norm = torch.ones(1, device=DEV)
    moe.moe_clip_grads([torch.empty(0, device=DEV)], 1.0, norm)
    assert norm.item() == 0.0


# ------------------------------------------------------- streams and captures
def test_other_stream_and_graph_replay():
    b = Batch(500, 64, 4, seqs=[0, 200, 480], masked=True, seed=21).device()
    b.run_loss()
    b.run_bwd()
    g = [torch.randn(4000, device=DEV), torch.randn(300, device=DEV).bfloat16()]
    kept = [t.clone() for t in g]
    out = [torch.empty_like(t) for t in g]
    lst, norm = moe.GradList(g, out), torch.empty(1, device=DEV)
    moe.moe_clip_grads(lst, 1.0, norm)
    want = [t.clone() for t in (b.loss, b.counts, b.mean, b.dlogits, norm, *out)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        b.run_loss(stream=torch.cuda.current_stream())
        b.run_bwd()
        moe.moe_clip_grads(lst, 1.0, norm)

    def same():
        torch.cuda.synchronize()
        for a, c in zip((b.loss, b.counts, b.mean, b.dlogits, norm, *out), want):
            assert torch.equal(a, c)
        for a, c in zip(g, kept):
            assert torch.equal(a, c)

    with torch.cuda.stream(side):
        step()
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (b.loss, b.dlogits, norm, *out):
        t.fill_(math.nan)
    for _ in range(3):
        graph.replay()
    same()
    clean(b.ws)


def test_binding_refuses_on_the_device():
    b = Batch(16, 8, 2).device()
    with pytest.raises(ValueError, match="shape"):
        moe.moe_balance_loss(b.dL[:, :4].contiguous(), b.didx, b.loss, b.counts, b.tokens, b.shape, b.ws)
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_balance_loss(b.dL.t().contiguous().t(), b.didx, b.loss, b.counts, b.tokens, b.shape, b.ws)
    with pytest.raises(TypeError, match="int32"):
        moe.moe_balance_loss(b.dL, b.didx.long(), b.loss, b.counts, b.tokens, b.shape, b.ws)
    with pytest.raises(ValueError, match="ws has"):
        moe.moe_balance_loss(b.dL, b.didx, b.loss, b.counts, b.tokens, b.shape, b.ws[:512])
    with pytest.raises(moe.MoEError):
        moe.moe_gate_bwd(b.dL, b.didx, b.dlogits, b.shape, b.ws)
    with pytest.raises(ValueError, match="contiguous"):
        moe.GradList([torch.zeros(8, 8, device=DEV).t()[1:]])

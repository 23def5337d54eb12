"""Training the gate at sizes whose offsets pass 32 bits, and with calls that run beside
one another.

The references are 64-bit torch products on the device, of all rows where a result sums
over them and of the first, the last and some other rows elsewhere.  u = 2^-24 is half a
step of fp32; the bounds are those of test_gpu_gate_train, with the length of the sums
as the library cuts them: at most 128 tokens on the tensor cores (three products each,
adds that may truncate, 2 u), then one fp32 add for each 128 tokens and for each
partial."""

import math

import pytest
import torch

import routing_dispatch_expert_softmax_b200 as moe
from routing_dispatch_expert_softmax_b200.binding import MoEShape

from parity_utils import U32

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
    torch.cuda.empty_cache()


def clean(ws):
    st = moe.moe_check(ws)
    assert st == moe.MOE_OK, moe.moe_error_string(st)


def some_rows(T):
    g = torch.Generator().manual_seed(T)
    return torch.cat([torch.arange(40), torch.arange(T - 40, T), torch.randint(0, T, (60,), generator=g)]).to(DEV)


def within(got, want, bound, name):
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), (name, float((off - bound).max()))


def check_router_large(x, W, dl, out):
    T, d = x.shape
    E = W.shape[1]
    n = 2 * (3 * 128 + 16) + T // 128 + 200
    cols = torch.cat([torch.arange(8), torch.arange(d - 8, d)]).to(DEV)
    want = torch.zeros(16, E, dtype=torch.float64, device=DEV)
    mags, db, dbm = torch.zeros_like(want), want.new_zeros(E), want.new_zeros(E)
    for t in range(0, T, 1 << 16):
        a, b = x[t:t + (1 << 16)][:, cols].double(), dl[t:t + (1 << 16)].double()
        want += a.t() @ b
        mags += a.abs().t() @ b.abs()
        db += b.sum(0)
        dbm += b.abs().sum(0)
    within(out["dw_g"][cols], want, n * U32 * mags, "dw_g")
    # a block adds up to T / 592 + 32 rows, then fp64 sums
    within(out["dbias"], db, (T // 592 + 50) * U32 * dbm, "dbias")
    rows = some_rows(T)
    l64, W64 = dl[rows].double(), W.double()
    ref, mag = l64 @ W64.t(), l64.abs() @ W64.abs().t()
    low = 2.0 ** -39 * (l64.abs().amax(1)[:, None] * W64.abs().sum(1)[None]
                        + l64.abs().sum(1)[:, None] * W64.abs().amax(1)[None])
    within(out["dx"][rows], ref, BF16 * ref.abs() + (1 + BF16) * (
        (2.0 ** -10 + 2.0 ** -22 + 2 * (E + 16) * U32) * mag + 1.01 * low) + 1e-37, "dx")


def router(T, d, E, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.empty(T, d, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    W = torch.randn(d, E, generator=g, device=DEV) / math.sqrt(d)
    dl = torch.randn(T, E, generator=g, device=DEV)
    s = MoEShape.of(T, d, E, 1, 64)
    out = dict(dw_g=torch.full((d, E), math.nan, device=DEV), dbias=torch.full((E,), math.nan, device=DEV),
               dx=torch.full((T, d), math.nan, dtype=torch.bfloat16, device=DEV))
    return x, W, dl, s, moe.workspace_bwd(s), out


@pytest.mark.parametrize("T,d,E", [(1 << 18, 8256, 8), (1 << 20, 64, 1024)])
def test_router_bwd_beyond_32_bits(T, d, E):
    # x and dx of more than 2^31 elements; planes of dlogits of as many
    x, W, dl, s, ws, out = router(T, d, E)
    moe.moe_router_bwd(x, W, dl, s, ws, **out)
    clean(ws)
    check_router_large(x, W, dl, out)


def test_combine_bwd_beyond_32_bits():
    T, d, k = 1 << 17, 2112, 8  # 2.2e9 elements of z
    g = torch.Generator(device=DEV).manual_seed(1)
    dy = torch.empty(T, d, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    z = torch.empty(T * k, d, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    row = torch.randperm(T * k, generator=g, device=DEV).int().view(T, k)
    w = torch.rand(T, k, generator=g, device=DEV)
    s = MoEShape.of(T, d, k, k, 64)
    dw = torch.full((T, k), math.nan, device=DEV)
    dz = torch.full((T * k, d), math.nan, dtype=torch.bfloat16, device=DEV)
    moe.moe_combine_bwd(dy, z, row, w, s, dw=dw, dz=dz)
    t = some_rows(T)
    r = row[t].long()
    prod = dy[t].double()[:, None, :] * z[r].double()
    within(dw[t], prod.sum(2), (d + 8) * 1.01 * U32 * prod.abs().sum(2), "dw")
    want = w[t].double()[:, :, None] * dy[t].double()[:, None, :]
    within(dz[r], want, (BF16 + 3 * U32) * want.abs(), "dz")
    assert not torch.isnan(dz[-1]).any() and not torch.isnan(dw).any()


def test_balance_and_gate_of_the_largest_batch():
    T, E, k, a, b = 1 << 20, 1024, 4, 0.02, 1e-3
    g = torch.Generator(device=DEV).manual_seed(2)
    L = torch.empty(T, E, device=DEV).normal_(generator=g)
    idx = torch.randint(0, E // k, (T, k), generator=g, device=DEV, dtype=torch.int32) * k
    idx += torch.arange(k, device=DEV, dtype=torch.int32)  # distinct in a token
    w, dw = torch.rand(T, k, generator=g, device=DEV), torch.randn(T, k, generator=g, device=DEV)
    seqs = torch.tensor([3, 5, T // 2, T - 1], dtype=torch.int32, device=DEV)
    s = MoEShape.of(T, 64, E, k, 64)
    ws = moe.workspace_bwd(s, 3)
    loss, counts = torch.empty(3, device=DEV), torch.empty(3, E, dtype=torch.int32, device=DEV)
    tokens, mean = torch.empty(5, dtype=torch.int32, device=DEV), torch.empty(3, E, device=DEV)
    moe.moe_balance_loss(L, idx, loss, counts, tokens, s, ws, a, b, seq_offsets=seqs, prob_mean=mean)
    dl = torch.full((T, E), math.nan, device=DEV)
    moe.moe_gate_bwd(L, idx, dl, s, ws, w=w, dw=dw, counts=counts, tokens=tokens, balance_coef=a,
                     z_coef=b, seq_offsets=seqs)
    clean(ws)
    off = seqs.tolist()
    n = [off[i + 1] - off[i] for i in range(3)]
    assert tokens.tolist() == [*n, sum(n), 3]
    psum = torch.zeros(3, E, dtype=torch.float64, device=DEV)
    z = 0.0
    for i in range(3):
        want = torch.bincount(idx[off[i]:off[i + 1]].flatten().long(), minlength=E)
        assert torch.equal(counts[i].long(), want)
        for t in range(off[i], off[i + 1], 1 << 16):
            q = L[t:min(off[i + 1], t + (1 << 16))].double()
            psum[i] += q.softmax(1).sum(0)
            z += float(q.logsumexp(1).square().sum())
    # |logits| < 6: differences of at most 12
    rel = (4.44 * 12 + E + 16 + -(-T // 296) + 44) * U32
    ref = psum / torch.tensor(n, device=DEV)[:, None]
    within(mean, ref, rel * ref, "prob_mean")
    bal = a / 3 * float(sum(E / (k * n[i]) * (counts[i].double() * ref[i]).sum() for i in range(3)))
    zl = b / sum(n) * z
    # lse ~ 7.4 is off by (2 lse + 6.1 + 6 log E) u and the sum's error, its square by twice that
    zrel = 2 * ((2 + 50 / 7) * U32 + (4.44 * 12 + E + 16) * U32 / 7) + (-(-T // 296) + 44) * U32
    assert abs(loss[1].item() - bal) <= (rel + 4 * U32) * bal
    assert abs(loss[2].item() - zl) <= zrel * zl
    rows = some_rows(T)
    p = L[rows].double().softmax(1)
    lse = L[rows].double().logsumexp(1)[:, None]
    seq = torch.bucketize(rows, seqs.long(), right=True) - 1
    live = ((seq >= 0) & (seq < 3)).double()[:, None]
    seq = seq.clamp(0, 2)
    nn = torch.tensor(n, device=DEV, dtype=torch.float64)[seq][:, None]
    f = a * E * counts[seq].double() / (3 * k * nn * nn)
    zc = 2 * b / sum(n) * lse
    dot = (f * p).sum(1, keepdim=True)
    want = live * p * (f - dot + zc)
    gw, gd = w[rows].double(), dw[rows].double()
    gate = gw * (gd - (gw * gd).sum(1, keepdim=True))
    want.scatter_add_(1, idx[rows].long(), gate)
    rel = (4.44 * 12 + E + 16) * U32
    dlse = U32 * (2 * lse + 6.1 + 6 * math.log(E)) + rel
    bound = live * p * ((rel + 12 * U32) * (f + dot + zc) + (rel + (E + 12) * U32) * dot
                        + 2 * b / sum(n) * dlse + 6 * U32 * zc)
    size = (gw * gd).abs()
    bound.scatter_add_(1, idx[rows].long(), U32 * ((k + 6) * size.sum(1, keepdim=True) * gw + 4 * size))
    within(dl[rows], want, bound + 2 * U32 * want.abs() + 1e-37, "dlogits")
    assert not torch.isnan(dl[-1]).any()


def test_clip_of_one_tensor_beyond_32_bits():
    n = (1 << 32) + 5
    g = torch.empty(n, dtype=torch.bfloat16, device=DEV)
    g.fill_(0.5)
    g[-7:] = 3.0
    norm = torch.empty(1, device=DEV)
    moe.moe_clip_grads([g], 1.0, norm)
    want = math.sqrt((n - 7) * 0.25 + 7 * 9.0)  # fp32 sums of 8 equal squares are exact
    assert abs(norm.item() - want) <= 2 * U32 * want
    c = 1.0 / (want + 1e-6)
    for part, v in ((g[:1000], 0.5), (g[n // 2:n // 2 + 1000], 0.5), (g[-1000:-7], 0.5), (g[-7:], 3.0)):
        assert bool(((part.double() - c * v).abs() <= (BF16 + 8 * U32) * c * v).all())


@pytest.mark.parametrize("T,d,E", [(20, 256, 40), (64, 4096, 128), (700, 512, 24), (2000, 256, 128)])
def test_router_bwd_on_two_streams_and_replayed(T, d, E):
    # calls on workspaces of their own may overlap; so may the graphs that hold them
    jobs, streams, graphs = [router(T, d, E, seed=i) for i in range(2)], [], []
    for x, W, dl, s, ws, out in jobs:
        moe.moe_router_bwd(x, W, dl, s, ws, **out)
    want = [{n: t.clone() for n, t in j[5].items()} for j in jobs]
    torch.cuda.synchronize()

    def same():
        torch.cuda.synchronize()
        for j, old in zip(jobs, want):
            clean(j[4])
            assert all(torch.equal(j[5][n], old[n]) for n in old)
            for t in j[5].values():
                t.fill_(math.nan)
        torch.cuda.synchronize()

    for x, W, dl, s, ws, out in jobs:
        st, gr = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            moe.moe_router_bwd(x, W, dl, s, ws, **out)
        streams.append(st), graphs.append(gr)
    for t in [t for j in jobs for t in j[5].values()]:
        t.fill_(math.nan)
    torch.cuda.synchronize()
    for _ in range(20):
        for (x, W, dl, s, ws, out), st in zip(jobs, streams):
            moe.moe_router_bwd(x, W, dl, s, ws, stream=st, **out)
    same()
    for _ in range(20):
        for st, gr in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
    same()

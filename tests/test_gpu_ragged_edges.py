"""Ragged-batch operators where their kernels and schedules change: weights in two parts,
prefixes over many ranges, places without a slot, data written right before a call.

Tolerances as derived in test_gpu_ragged.py, for weights of two bf16 parts: the low part
is off by 2^-8 of what the high part left, 2^-8 of the weight, so 2^-16 together.  Both
parts' products are added in fp32, 2 n additions over n keys:
  |err| <= 2^-8 |out| (1 + w) + w sum p|v|,  w = 260 u A + 2^-16 + 2^-19 + 2 n u.
Append: beside the roundings of the two products, the angle, below 2 pi, is rounded to fp32
(at most 2^-22 = 4 u off), and a sine or cosine moves by as much whatever its own size, as it
does by the function's error (below 4 u): 8 u of each unrotated value, near a zero of the
cosine far more than 64 u of the product.
"""
import threading

import pytest
import torch

import ragged_ref as ref
import speculative_decoding_fc_gb300 as ds
from test_gpu_ragged import HD, U, _gen, _hide, _lens, _normal

pytestmark = pytest.mark.gpu


def _close2(out, want, av, a, n):
    w = 260 * U * a + 2.0 ** -16 + 2.0 ** -19 + 2 * n * U
    bound = 2.0 ** -8 * want.abs() * (1 + w) + w * av + 1e-30
    assert torch.isfinite(out).all()
    worst = ((out.double() - want).abs() / bound).max().item()
    assert worst <= 1.0, "error %.3g of the bound" % worst


PARTS_CASES = [
    # nr, nq, nkv, cache, lens, window, sinks, causal: 17 to 64 rows per kv head
    (8, 40, 8, 1100, [1032, 8, 5, 0], 512, 4, False),
    (8, 40, 8, 5000, [4999, 2500, 129, 8], 0, 0, True),
    (17, 4, 4, 300, [300, 64, 63, 65, 1], 0, 0, True),
    (64, 2, 2, 700, [699, 64, 128], 33, 70, True),
    (1, 40, 1, 2000, [2000, 1], 0, 0, False),
]


@pytest.mark.parametrize("case", range(len(PARTS_CASES)))
def test_weights_of_blocks_have_two_parts(case):
    nr, nq, nkv, cache, lens, window, sinks, causal = PARTS_CASES[case]
    g = _gen(1000 + case)
    B = len(lens)
    q = _normal((B, nr, nq, HD), g, 1.5)
    kc, vc = _normal((B, cache, nkv, HD), g), _normal((B, cache, nkv, HD), g)
    _hide(kc, vc, nr, lens, window, sinks, causal)
    want, av, a = ref.window(q, kc, vc, lens, window, sinks, causal)
    _close2(ds.window_attention(q, kc, vc, _lens(lens), window, sinks=sinks, causal=causal), want, av, a, cache)
    if not window:
        _close2(ds.attention_scored(q, kc, vc, _lens(lens), causal=causal)[0], want, av, a, cache)


PREFIX_CASES = [
    # B, nr, nq, nkv, P, cache, lens, causal
    (3, 1, 40, 8, 4096, 70, [0, 64, 70], True),            # 15 rows: the decode kernel, many ranges
    (1, 2, 40, 8, 1025, 70, [2], False),
    (2, 1, 40, 8, 20000, 130, [130, 0], True),             # ... with the cost of changing items
    (1, 1, 16, 1, 3333, 65, [65], True),
    (4, 1, 40, 8, 4096, 70, [0, 1, 64, 70], True),         # 20 rows: tcgen05, four warps to a row in the join
    (1, 8, 40, 8, 20000, 130, [130], True),
    (1, 8, 40, 8, 20000, 130, [0], False),
    (12, 1, 40, 8, 1031, 300, [25 * b for b in range(12)], True),   # 60 rows
    (64, 1, 8, 8, 2500, 70, [(9 * b) % 71 for b in range(64)], True),
]


@pytest.mark.parametrize("case", range(len(PREFIX_CASES)))
def test_few_rows_over_a_long_prefix(case):
    B, nr, nq, nkv, P, cache, lens, causal = PREFIX_CASES[case]
    g = _gen(1100 + case)
    q = _normal((B, nr, nq, HD), g, 1.5)
    kp, vp = _normal((P, nkv, HD), g), _normal((P, nkv, HD), g)
    kc, vc = _normal((B, cache, nkv, HD), g), _normal((B, cache, nkv, HD), g)
    _hide(kc, vc, nr, lens, 0, 0, causal)
    want, av, a = ref.prefix(q, kp, vp, kc, vc, lens, causal)
    out = ds.shared_prefix_attention(q, kp, vp, kc, vc, _lens(lens), causal=causal)
    _close2(out, want, av, a, P + cache)
    assert torch.equal(out, ds.shared_prefix_attention(q, kp, vp, kc, vc, _lens(lens), causal=causal))


@pytest.mark.parametrize("P", [500, 4096, 20000])
def test_prefix_schedule_found_by_warps_and_by_the_plan(P):
    """32 requests (each warp works its range out) and the same with an empty one behind them
    (the plan kernel does): the same kernel and ranges, so the same bits."""
    g = _gen(1200 + P)
    B, n, nkv, cache = 33, 32, 8, 90
    lens = [(13 * b * b + 7) % 91 for b in range(n)] + [0]
    q = _normal((B, 1, nkv, HD), g, 1.5)
    kp, vp = _normal((P, nkv, HD), g), _normal((P, nkv, HD), g)
    kc, vc = _normal((B, cache, nkv, HD), g), _normal((B, cache, nkv, HD), g)
    want, av, a = ref.prefix(q, kp, vp, kc, vc, lens, True)
    full = ds.shared_prefix_attention(q, kp, vp, kc, vc, _lens(lens), causal=True)
    _close2(full, want, av, a, P + cache)
    assert torch.equal(full[:n], ds.shared_prefix_attention(q[:n], kp, vp, kc[:n], vc[:n], _lens(lens[:n]), causal=True))


@pytest.mark.parametrize("B,nr", [(3, 1), (6, 1), (40, 8), (6, 8)])
def test_lengths_out_of_range_with_a_prefix_and_with_scores(B, nr):
    g = _gen(1300 + B + nr)
    nq, nkv, cache, P = 40, 8, 80, 600
    q = _normal((B, nr, nq, HD), g)
    kp, vp = _normal((P, nkv, HD), g), _normal((P, nkv, HD), g)
    kc, vc = _normal((B, cache, nkv, HD), g), _normal((B, cache, nkv, HD), g)
    for bad in (-1, cache + 1):
        lens = [(11 * b + 3) % (cache + 1) for b in range(B)]
        lens[B - 2] = bad
        good = [min(max(n, 0), cache) for n in lens]
        spaces = ds.Workspaces()
        out = ds.shared_prefix_attention(q, kp, vp, kc, vc, _lens(lens), workspaces=spaces)
        assert ds.workspace_status(spaces.buffer("ragged_prefix", q.device)) == -1
        assert torch.equal(out, ds.shared_prefix_attention(q, kp, vp, kc, vc, _lens(good), workspaces=spaces))
        assert ds.workspace_status(spaces.buffer("ragged_prefix", q.device)) == 0
        sc = torch.rand((B, nkv, cache), device="cuda", generator=g)
        out, new = ds.attention_scored(q, kc, vc, _lens(lens), sc.clone(), workspaces=spaces)
        assert ds.workspace_status(spaces.buffer("ragged_scored", q.device)) == -1
        out1, new1 = ds.attention_scored(q, kc, vc, _lens(good), sc.clone(), workspaces=spaces)
        assert torch.equal(out, out1) and torch.equal(new, new1)
        assert ds.workspace_status(spaces.buffer("ragged_scored", q.device)) == 0


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("B,nr,nq,nkv,P,cache", [(16, 8, 40, 8, 1500, 600), (80, 1, 20, 4, 3000, 300)])
def test_shared_prefix_of_data_written_right_before(B, nr, nq, nkv, P, cache, graph):
    """The launch over the own keys starts beside the prefix's: q, the lengths, the prefix and
    the caches, written on the device directly before each call, are the call's."""
    g = _gen(1400 + B)
    bufs = [torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in
            ((B, nr, nq, HD), (P, nkv, HD), (P, nkv, HD), (B, cache, nkv, HD), (B, cache, nkv, HD))]
    lens = torch.empty(B, dtype=torch.int32, device="cuda")
    sets, want = [], []
    for i in range(4):
        new = [_normal(b.shape, g, 1.5) for b in bufs]
        n = _lens([(31 * b + 17 * i * i) % (cache + 1) for b in range(B)])
        sets.append((new, n))
        torch.cuda.synchronize()
        want.append(ds.shared_prefix_attention(new[0], *new[1:], n, causal=True))
        torch.cuda.synchronize()

    def step(new, n):
        for b, x in zip(reversed(bufs), reversed(new)):   # q last
            torch.mul(x, 1.0, out=b)
        torch.mul(n, 1, out=lens)
        return ds.shared_prefix_attention(bufs[0], *bufs[1:], lens, causal=True)

    def rounds():
        return [step(*sets[i % 4]) for i in range(8)]

    got = rounds()
    if graph:
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            got = rounds()
        captured.replay()
        captured.replay()
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        assert torch.equal(x, want[i % 4])


def _rotated_close(got, x, w, at):
    want, mag = ref.rope(x, w, at, 1e6)
    y = x.double()
    y = (y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.double()).abs()
    pair = y[..., :64] + y[..., 64:]
    bound = 2.0 ** -8 * want.abs() + 64 * U * mag + 8 * U * torch.cat([pair, pair], -1)
    assert ((got.double() - want).abs() <= bound).all()


def test_negative_position_without_slots():
    """No slot given: a request at a negative position has none, and nothing of it is stored."""
    g = _gen(1500)
    B, rows, nq, nkv, cache = 3, 8, 4, 2, 32
    kc, vc = _normal((B, cache, nkv, HD), g), _normal((B, cache, nkv, HD), g)
    k0, v0 = kc.clone(), vc.clone()
    qkv = _normal((B * rows, (nq + 2 * nkv) * HD), g)
    w = torch.ones(HD, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = [5, -3, 2]
    q = ds.qk_norm_rope_ragged(qkv, nq, nkv, w, w, 1e6, kc, vc, rows, _lens(pos), status=st)
    assert int(st.item()) == -1
    assert torch.equal(kc[1], k0[1]) and torch.equal(vc[1], v0[1])
    x = qkv.view(B, rows, nq + 2 * nkv, HD)
    for b, p in enumerate([5, 0, 2]):   # queries: a negative position counts as 0
        at = torch.arange(rows, device="cuda") + p
        _rotated_close(q.view(B, rows, nq, HD)[b], x[b, :, :nq], w, at)
        if b != 1:
            _rotated_close(kc[b, p:p + rows], x[b, :, nq:nq + nkv], w, at)
            assert torch.equal(vc[b, p:p + rows], x[b, :, nq + nkv:])


def test_overlapping_outputs_are_refused():
    g = _gen(1600)
    q, kc, vc = _normal((2, 4, 8, HD), g), _normal((2, 64, 8, HD), g), _normal((2, 64, 8, HD), g)
    lens, sc = _lens([64, 9]), torch.zeros((2, 8, 64), device="cuda")
    w = torch.ones(HD, dtype=torch.bfloat16, device="cuda")
    wide = _normal((9, 24 * HD), g)   # its first 8 rows are the call's
    two = torch.zeros((3, 8, 64), device="cuda")
    for call in (lambda: ds.window_attention(q, kc, vc, lens, 0, out=q),
                 lambda: ds.window_attention(q, kc, vc, lens, 0, out=vc.view(-1)[:q.numel()].view(q.shape)),
                 lambda: ds.shared_prefix_attention(q, q[0], vc[0, :4], kc, vc, lens, out=q),
                 lambda: ds.shared_prefix_attention(q, kc[0], wide[:4, :8 * HD].reshape(4, 8, HD), kc, vc, lens,
                                                    out=vc.view(-1)[8 * HD:8 * HD + q.numel()].view(q.shape)),
                 lambda: ds.attention_scored(q, kc, vc, lens, sc, out=q),
                 lambda: ds.attention_scored(q, kc, vc, lens, two[:2], scores_out=two[1:]),
                 lambda: ds.qk_norm_rope_ragged(wide[:8], 8, 8, w, w, 1e6, kc, kc, 4, lens),
                 lambda: ds.qk_norm_rope_ragged(wide[:8], 8, 8, w, w, 1e6, kc, vc, 4, lens,
                                                q_out=wide.view(-1)[HD:HD + 64 * HD].view(8, 8, HD))):
        with pytest.raises(ValueError, match="overlap"):
            call()
    # right behind one another is apart
    both = torch.empty((2,) + q.shape, dtype=torch.bfloat16, device="cuda")
    both[0] = q
    got = ds.window_attention(both[0], kc, vc, lens, 0, out=both[1])
    assert torch.equal(got, ds.window_attention(q, kc, vc, lens, 0)) and torch.equal(both[0], q)
    assert ds.attention_scored(q, kc, vc, lens, sc, scores_out=sc)[1] is sc


def test_calls_from_two_threads():
    """Host threads with streams and workspaces of their own, each form and the append."""
    g = _gen(1700)
    w = torch.ones(HD, dtype=torch.bfloat16, device="cuda")
    sets = []
    for i in range(2):
        kc, vc = _normal((4, 300, 4, HD), g), _normal((4, 300, 4, HD), g)
        sets.append((kc, vc, _lens([300, 1, 64 + i, 200]), [_normal((4, n, 8, HD), g) for n in (1, 9, 40)],
                     _normal((32, 16 * HD), g), torch.zeros((2, 4, 320, 4, HD), dtype=torch.bfloat16, device="cuda")))
    torch.cuda.synchronize()

    def work(i, stream, spaces, got):
        kc, vc, lens, qs, qkv, new = sets[i]
        for _ in range(3):
            for q in qs:
                got.append(ds.window_attention(q, kc, vc, lens, 0, stream=stream, workspaces=spaces))
                got.append(ds.shared_prefix_attention(q, kc[0], vc[0], kc, vc, lens, stream=stream, workspaces=spaces))
                if q.shape[1] < 32:
                    got.extend(ds.attention_scored(q, kc, vc, lens, stream=stream, workspaces=spaces))
            got.append(ds.qk_norm_rope_ragged(qkv, 8, 4, w, w, 1e6, new[0], new[1], 8, lens, stream=stream))

    want, got, failed = [[], []], [[], []], []
    for i in range(2):
        work(i, torch.cuda.Stream(), ds.Workspaces(), want[i])
        torch.cuda.synchronize()

    def run(i):
        try:
            work(i, torch.cuda.Stream(), ds.Workspaces(), got[i])
        except Exception as e:   # (a thread's exception would be lost)
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for i in range(2):
        assert len(got[i]) == len(want[i])
        for x, y in zip(got[i], want[i]):
            assert torch.equal(x, y)


def test_append_over_far_positions():
    """Many rows at positions up to a million: some pairs stand where the cosine is near zero."""
    g = _gen(1800)
    B, rows, nq, nkv = 200, 9, 20, 4
    kc, vc = (torch.zeros((B, rows, nkv, HD), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qkv = _normal((B * rows, (nq + 2 * nkv) * HD), g, 2.0)
    w = (1.0 + _normal((HD,), g, 0.1, torch.float32)).bfloat16()
    pos = [(4999 * b * b + 17 * b) % 1000003 for b in range(B)]
    q = ds.qk_norm_rope_ragged(qkv, nq, nkv, w, w, 1e6, kc, vc, rows, _lens(pos), slot=_lens([0] * B))
    at = (_lens(pos)[:, None] + torch.arange(rows, device="cuda")).view(-1)
    x = qkv.view(B * rows, nq + 2 * nkv, HD)
    _rotated_close(q, x[:, :nq], w, at)
    _rotated_close(kc.view(B * rows, nkv, HD), x[:, nq:nq + nkv], w, at)
    assert torch.equal(vc.view(B * rows, nkv, HD), x[:, nq + nkv:])

"""GPU parity of the verification of drafted tokens (qmm_serve.h) with oracle/serve_oracle.py: tokens are equal."""
import numpy as np
import pytest
import torch

import gemm_affine_u4_amd as qmm
from oracle import serve_oracle as srv
from tests.gpu_util import dev
from tests.serve_util import bf16, ints

pytestmark = pytest.mark.gpu


def call(draft, start, target, q, u, max_draft, half, at=0):
    """One call with guarded outputs; probabilities start `at` elements into their buffers."""
    B = len(start) - 1

    def put(x):
        flat = dev(bf16(x)[0].ravel()).view(torch.bfloat16) if half else dev(x.astype(np.float32).ravel())
        buf = torch.full((flat.numel() + 64,), float("nan"), dtype=flat.dtype, device="cuda")
        buf[at:at + flat.numel()] = flat
        return buf[at:at + flat.numel()].view(x.shape)

    tokens = torch.full((B + 2, max_draft + 1), -77, dtype=torch.int32, device="cuda")
    accepted = torch.full((B + 2,), -77, dtype=torch.int32, device="cuda")
    ws = torch.full((qmm.qmm_spec_verify_workspace_bytes(B, target.shape[1]) + 512,), 255, dtype=torch.uint8, device="cuda")
    qmm.qmm_spec_verify(dev(draft.astype(np.int32)), put(target), dev(u.astype(np.float32)), tokens[1:-1], accepted[1:-1],
                        ws[:-512], dev(start.astype(np.int32)), draft_probs=None if q is None else put(q))
    torch.cuda.synchronize()
    assert bool((tokens[[0, -1]] == -77).all()) and bool((accepted[[0, -1]] == -77).all())
    assert bool((ws[-512:] == 255).all())
    return tokens[1:-1].cpu().numpy(), accepted[1:-1].cpu().numpy()


def held(x, half):
    return bf16(x)[1] if half else x.astype(np.float32).astype(np.float64)


def check(rng, counts, V, probs, half, at=0, sharp=3.0, max_draft=None):
    B, D = len(counts), int(np.sum(counts))
    start = np.concatenate([[0], np.cumsum(counts)])
    logits = sharp * rng.standard_normal((D + B, V))
    target = np.exp(logits - logits.max(1, keepdims=True))
    target /= target.sum(1, keepdims=True)
    rows = np.array([start[b] + b + j for b in range(B) for j in range(counts[b])], int)
    other = np.exp(0.4 * rng.standard_normal((D, V))) * target[rows]
    other /= other.sum(1, keepdims=True)
    draft = np.array([rng.choice(V, p=x) for x in other], int).reshape(D)
    target, other = held(target, half), held(other, half)
    u = rng.random(D + B).astype(np.float32)
    max_draft = max(max(counts), 0) if max_draft is None else max_draft
    got = call(draft, start, target, other if probs else None, u, max_draft, half, at)
    want = srv.verify(draft, start, target, other if probs else None, u, max_draft)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])
    return want


@pytest.mark.parametrize("V", [1, 2, 63, 1000, 4096, 4097, 32003, 131072])
@pytest.mark.parametrize("probs,half", [(True, False), (False, False), (True, True), (False, True)])
def test_batches(V, probs, half):
    rng = np.random.default_rng([V, probs, half])
    tokens, acc = check(rng, [3, 0, 5, 1, 2, 7, 4], V, probs, half)
    check(rng, [0], V, probs, half)
    check(rng, [6], V, probs, half, at=1)  # probabilities at an odd address
    if V > 1000 and probs:
        assert acc.max() > 0


@pytest.mark.parametrize("V", [16383, 16384, 16385, 24576])
@pytest.mark.parametrize("half", [False, True])
def test_where_rows_take_two_launches(V, half):
    rng = np.random.default_rng([9, V, half])
    for at in (0, 3):
        check(rng, [2, 0, 4, 1], V, True, half, at=at)
        check(rng, [1, 3], V, False, half, at=at)


def test_many_sequences_and_a_long_draft():
    rng = np.random.default_rng(1)
    tokens, acc = check(rng, rng.integers(0, 5, 300).tolist(), 500, True, False)
    assert 0 < (acc == 0).sum() < 300
    check(rng, [600, 3], 40, True, False, sharp=0.1)
    check(rng, [9, 2, 4], 300, True, False, max_draft=3)  # drafts past max_draft do not count
    check(rng, [2, 1], 300, True, False, max_draft=6)


def test_all_kept_and_where_the_first_is_refused():
    rng = np.random.default_rng(2)
    V, n = 700, 300
    start, draft = np.array([0, n]), rng.integers(0, V, n)
    p = np.full((n + 1, V), 1.0 / V)
    q = np.full((n, V), 2.0 / V)      # kept while u < 1/2
    for at in (0, 1, 63, 64, 255, 256, 257, n - 1, n):
        u = np.full(n + 1, 0.25)
        u[at:n] = rng.choice([0.25, 0.75], n - at)
        u[at] = 0.75
        got, want = call(draft, start, p, q, u, n, False), srv.verify(draft, start, held(p, 0), held(q, 0), u, n)
        assert got[1][0] == at and np.array_equal(got[0], want[0])


@pytest.mark.parametrize("probs", [True, False])
def test_corners(probs):
    """No such token, rows of zeros, p equal to q, one-hot rows, numbers at the ends, weights NaN and below 0."""
    rng = np.random.default_rng(3)
    V = 5000
    p = rng.random((14, V))
    p /= p.sum(1, keepdims=True)
    q = p[:7] * rng.uniform(0.5, 1.5, (7, V))
    draft = rng.integers(0, V, 7)
    start = np.arange(8)
    p[2 * 0] = 0
    p[2 * 1], q[1] = p[3], p[3]                  # nothing is left where it is refused
    draft[1] = -1
    draft[2] = V
    p[2 * 3] = 0
    p[2 * 3, V - 1] = 1.0                         # one-hot, at the end
    p[2 * 4 + 1] = 0                              # a new token of a row of zeros
    draft[4], p[2 * 4, draft[4]], q[4, draft[4]] = 17, 0.9, 0.3
    p[2 * 5, ::3] = np.nan
    p[2 * 5, 1::3] = -1.0
    draft[5] = 0
    p[2 * 6] = 0
    p[2 * 6, 4095:4097] = 0.5                     # the weights lie on both sides of a chunk's end
    p, q = held(p, False), held(q, False)
    draft[6] = 11
    for numbers in ([0.0, 0.0], [0.5, 0.5], [0.999, np.float32(1 - 2.0 ** -24)], [0.3, 1.0], [0.9, -0.5]):
        u = np.tile(np.array(numbers, np.float32), 7)
        got, want = call(draft, start, p, q if probs else None, u, 1, False), srv.verify(
            draft, start, p, q if probs else None, u, 1)
        assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0]), numbers


def test_no_drafts_at_all():
    rng = np.random.default_rng(4)
    p = held(rng.dirichlet(np.ones(100), 3), False)
    u = rng.random(3).astype(np.float32)
    got, want = call(np.zeros(0), np.zeros(4), p, None, u, 0, False), srv.verify(np.zeros(0), np.zeros(4), p, None, u, 0)
    assert np.array_equal(got[0], want[0]) and np.all(got[1] == 0)


def test_starts_out_of_order_stay_inside():
    """Starts that fall or leave [0, D] are held inside it: such a sequence has no drafts, the others theirs."""
    rng = np.random.default_rng(5)
    p, q = held(rng.dirichlet(np.ones(50), 9), False), held(rng.dirichlet(np.ones(50), 5), False)
    u = rng.random(9).astype(np.float32)
    got = call(rng.integers(0, 50, 5), np.array([0, 2, 1, 99, 4]), p, q, u, 4, False)
    assert got[1].shape == (4,) and np.all((got[0] >= -1) & (got[0] < 50))


def test_in_a_graph():
    rng = np.random.default_rng(6)
    V, counts = 9000, [4, 2, 3]
    start = np.concatenate([[0], np.cumsum(counts)])
    p, q = rng.dirichlet(np.ones(V), 12).astype(np.float32), rng.dirichlet(np.ones(V), 9).astype(np.float32)
    draft, u = rng.integers(0, V, 9), rng.random(12).astype(np.float32)
    dp, dq, dd, du, ds = dev(p), dev(q), dev(draft.astype(np.int32)), dev(u), dev(start.astype(np.int32))
    graphs = []
    for _ in range(2):
        tokens = torch.empty(3, 5, dtype=torch.int32, device="cuda")
        acc = torch.empty(3, dtype=torch.int32, device="cuda")
        ws = torch.empty(qmm.qmm_spec_verify_workspace_bytes(3, V), dtype=torch.uint8, device="cuda")

        def run():
            qmm.qmm_spec_verify(dd, dp, du, tokens, acc, ws, ds, draft_probs=dq)

        run()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            run()
        graphs.append((gr, tokens, acc, ws))
    for seed in range(4):  # new numbers, read on the device
        u = np.random.default_rng(seed).random(12).astype(np.float32) * (0.2 if seed % 2 else 1.0)
        du.copy_(torch.from_numpy(u))
        want = srv.verify(draft, start, p, q, u, 4)
        for gr, tokens, acc, ws in graphs:
            ws.fill_(255)
            gr.replay()
        torch.cuda.synchronize()
        for gr, tokens, acc, ws in graphs:
            assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(acc.cpu().numpy(), want[1])


def test_frequencies():
    """Kept drafts and new tokens of many sequences have the target's frequencies."""
    rng = np.random.default_rng(7)
    V, N = 6, 30000
    p, q = held(rng.dirichlet(np.ones(V)), False), held(rng.dirichlet(np.ones(V)), False)
    draft = rng.choice(V, N, p=q / q.sum())
    got, acc = call(draft, np.arange(N + 1), np.tile(p, (2 * N, 1)), np.tile(q, (N, 1)), rng.random(2 * N), 1, False)
    # a frequency's deviation is at most 1/2 / sqrt(N): five of them
    assert np.abs(np.bincount(got[:, 0], minlength=V) / N - p).max() < 2.5 / np.sqrt(N)
    assert np.array_equal(acc == 1, got[:, 1] >= 0)

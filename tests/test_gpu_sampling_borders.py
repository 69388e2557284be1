"""The sampled token where the random number meets a border between running
sums, which the parts of a row add up in different orders."""
import numpy as np
import pytest
import torch

from decode_megakernel_interpreter_b200 import serving as sv

pytestmark = pytest.mark.gpu

# A running sum is off by at most this much of the row's: fewer than 64
# additions (a lane's values, trees over lanes, segments, blocks) lie between a
# weight and the sum, plus the product u * sum, each half a unit of 2^-53.
EPS = 64 * 2.0 ** -53


def sample(p, u):
    """New tokens of the rows p (numpy float32 [rows][vocab]), u one number or one a row."""
    n = p.shape[0]
    u = torch.full((n, 1), 0.0, device="cuda") + torch.as_tensor(u, dtype=torch.float32, device="cuda").reshape(-1, 1)
    tok, acc = sv.verify(torch.from_numpy(p).cuda().unsqueeze(1), None, torch.zeros(n, 0, dtype=torch.int32, device="cuda"),
                         u.contiguous())
    assert (acc == 0).all()
    return tok[:, 0].tolist(), u[:, 0].double().tolist()


def check(p, u):
    """A token of weight above 0 at which the exact running sum passes u * sum, but for EPS."""
    toks, us = sample(p, u)
    for row, i, x in zip(p, toks, us):
        assert 0 <= i < len(row) and row[i] > 0, (i, x)
        at = np.flatnonzero(row)
        w = [int(v * 2.0 ** 149) for v in row[at].astype(np.float64)]  # exact
        k, total = int(np.searchsorted(at, i)), sum(w)
        goal, slack = x * total, EPS * total
        assert sum(w[:k + 1]) >= goal - slack and sum(w[:k]) <= goal + slack, (i, x)


def test_a_goal_between_two_blocks_sums():
    p = np.zeros((1, 50001), np.float32)
    p[0, [3584, 6656]] = 0.5
    p[0, [4096, 6144]] = 2.0 ** -54
    check(p, 0.5)


def test_a_goal_that_a_segment_without_weight_would_pass():
    p = np.zeros((1, 128256), np.float32)
    p[0, [3584, 20000]] = 0.5
    p[0, [4096, 6144]] = 2.0 ** -54
    check(p, 0.5)


@pytest.mark.parametrize("V", [513, 4097, 32003, 50001, 128256, 151936])
def test_goals_on_borders(V):
    """Two heavy tokens with weights next to the last bit of their sum scattered around them, the goal on the border."""
    r = np.random.RandomState(V)
    p = np.zeros((256, V), np.float32)
    u = np.zeros(256)
    for row in range(256):
        at = np.sort(r.choice(V, 2, replace=False))
        a = int(r.randint(1, 64))
        tiny = r.choice(V, min(V // 4, int(r.randint(1, 40))), replace=False)
        p[row, tiny] = 2.0 ** -r.randint(53, 58, len(tiny))
        p[row, at] = a / 64, 1 - a / 64
        u[row] = a / 64
    check(p, u)


@pytest.mark.parametrize("V", [50257, 100000])
def test_residuals_on_borders(V):
    """The same where the weights are what p exceeds q by."""
    r = np.random.RandomState(V)
    n = 128
    p, q = np.zeros((n, 2, V), np.float32), np.zeros((n, 1, V), np.float32)
    w = np.zeros((n, V), np.float32)
    u = np.zeros((n, 2), np.float32)
    for row in range(n):
        at = np.sort(r.choice(V, 3, replace=False))
        tiny = r.choice(V, 30, replace=False)
        w[row, tiny] = 2.0 ** -r.randint(55, 60, len(tiny))
        w[row, at[:2]] = 0.125
        w[row, at[2]] = 0
        q[row, 0, at] = 0.125, 0.25, 0.5
        p[row, 0] = w[row]
        p[row, 0, at] += q[row, 0, at]
        p[row, 0, at[2]] = 0.25
        w[row] = np.maximum(p[row, 0] - q[row, 0], 0)
        u[row] = 0.75, 0.5  # the token at[2] is refused: 0.75 * 0.5 is not below 0.25
    x = torch.from_numpy(q[:, 0].argmax(1).astype(np.int32)).cuda().reshape(n, 1)
    tok, acc = sv.verify(torch.from_numpy(p).cuda(), torch.from_numpy(q).cuda(), x, torch.from_numpy(u).cuda())
    assert (acc == 0).all()
    for row, i in enumerate(tok[:, 0].tolist()):
        at = np.flatnonzero(w[row])
        assert 0 <= i < V and w[row, i] > 0, i
        v = [int(y * 2.0 ** 149) for y in w[row, at].astype(np.float64)]
        k, total = int(np.searchsorted(at, i)), sum(v)
        assert sum(v[:k + 1]) >= 0.5 * total - EPS * total and sum(v[:k]) <= 0.5 * total + EPS * total, i


def test_the_largest_vocabulary():
    """104857600 tokens: weights in a few places; the additions of a block's 25600 segments are 800 more."""
    V = 104857600
    at = [0, 511, 512, 13107199, 13107200, 60000001, 104857088, 104857599]
    w = [3, 1, 4, 1, 5, 9, 2, 6]
    p = torch.zeros(1, 1, V, device="cuda")
    p[0, 0, at] = torch.tensor(w, dtype=torch.float32, device="cuda") / 32
    for u in np.linspace(0, 0.999, 23).astype(np.float32):  # (exact sums)
        tok, acc = sv.verify(p, None, torch.zeros(1, 0, dtype=torch.int32, device="cuda"), torch.tensor([[float(u)]], device="cuda"))
        assert tok.item() == at[int(np.argmax(np.cumsum(w) > float(u) * sum(w)))] and acc.item() == 0
    p.uniform_()
    total = p.double().sum()
    tok, acc = sv.verify(p, None, torch.zeros(1, 0, dtype=torch.int32, device="cuda"), torch.tensor([[0.7]], device="cuda"))
    i, goal, slack = tok.item(), float(np.float32(0.7)) * float(total), (64 + 800) * 2.0 ** -53 * float(total)
    c = p[0, 0, :i + 1].double().cumsum(0)  # (its own additions, as many as tokens, are off by V 2^-53 at most)
    assert c[i] >= goal - slack - V * 2.0 ** -53 * float(total) and c[i - 1] <= goal + slack + V * 2.0 ** -53 * float(total)

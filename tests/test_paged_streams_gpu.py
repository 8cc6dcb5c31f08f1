"""Sessions on a stream of their own while the current one is busy: nothing that a session makes or
copies for itself may come late."""
import pytest
import torch

import paged_ref as P
import test_paged_gpu as T
from adaptive_head_kv_gb300 import fastgen as fg
from adaptive_head_kv_gb300.session import PagedSession, make_params

pytestmark = pytest.mark.gpu

L, H, N, D = 2, 4, 150, 64
BUSY = 200_000_000  # cycles, a tenth of a second


def inputs(seed, *shape):
    return T.dev(torch.randn(*shape, generator=T.gen(seed)).to(torch.bfloat16))


def prompt(stream=None):
    p = make_params(1, L, H, N, D, "bf16", 0.9, 0.3, 0.3)
    s = PagedSession(p, T.SPECIAL, T.PUNCT, 8, rope=fg.Rope(T.table(D)[1]), stream=stream)
    ids = torch.randint(100, 300, (1, N), generator=T.gen(1), dtype=torch.int32)
    given = [inputs(x, L * H, N, D) for x in (2, 3, 4)] + [T.dev(ids)]
    torch.cuda.synchronize()
    return s, given, torch.arange(L * H, dtype=torch.int8) % 5


def rows(s):
    gpu, out = P.GpuPages(s.cache), []
    for c in range(s.Gkv):
        for ring, count in ((False, int(gpu.rows[c])), (True, int(gpu.caches[c][1]))):
            out += [x.tolist() for x in gpu.segment(c, ring, count).values()] if count else []
    return out


@pytest.mark.parametrize("as_address", [False, True])
def test_a_fork_made_while_the_current_stream_is_busy(as_address):
    side = torch.cuda.Stream()
    s, given, policies = prompt(side.cuda_stream if as_address else side)
    s.prefill_with_policy(*given, policies)
    torch.cuda.synchronize()
    B, forks, outs = 3, [], []
    steps = [[inputs(10 * st + x, B * L * H, D) for x in range(3)]
             + [T.dev([5, 1, 11], torch.int32), T.dev([N + st] * B, torch.int32)]
             for st in range(20)]
    for busy in (False, True):
        torch.cuda.synchronize()
        if busy:
            torch.cuda._sleep(BUSY)
        f = s.fork(B, 30, budget=16, recent=4, guard=True)
        out = [torch.empty_like(steps[0][0]) for _ in steps]
        for x, y in zip(steps, out):
            f.decode(*x, out=y)
        f.evict(steps[-1][-1])
        torch.cuda.synchronize()
        assert fg.fastgen_read_error(f.dev_err) == fg.FG_OK and f.check_guards() == 0
        forks.append(f)
        outs.append(torch.stack(out))
    assert torch.equal(*outs) and float(outs[0].abs().max()) > 0
    assert rows(forks[0]) == rows(forks[1])


def test_a_saved_policy_map_while_the_current_stream_is_busy():
    got = []
    for stream in (None, torch.cuda.Stream()):
        s, given, policies = prompt(stream)
        if stream is not None:
            torch.cuda._sleep(BUSY)
        s.prefill_with_policy(*given, policies)
        torch.cuda.synchronize()
        assert s.policy.tolist() == policies.tolist()
        assert fg.fastgen_read_error(s.dev_err) == fg.FG_OK
        got.append(rows(s))
    assert got[0] == got[1]

"""DropoutCounter and FlashDropout without a GPU: keys in recomputed functions
(activation checkpointing), between threads and in copies of a module.  Masks
come from the oracle, so any wrong key is a wrong gradient here."""

import copy
import threading
import time

import pytest
import torch
from torch.utils.checkpoint import checkpoint

from oracle import rows as R
from precision_optimizer_state_amd import nn


def drop(x, key, p=0.5):
    """What nn.dropout computes, in torch operations on the CPU."""
    keep = torch.from_numpy(R.keep(*x.shape, p, key["seed"], key["offset"]))
    return torch.where(keep, x * R.scale(p), torch.zeros_like(x))


@pytest.mark.parametrize("reentrant", [True, False])
@pytest.mark.parametrize("noise", [False, True])
def test_recomputed_segments_find_their_masks(reentrant, noise):
    """Three segments of two dropouts each; with `noise` they draw from torch's generator too.
    The masks are linear, so the gradient of x is the product of the masks and scales."""
    counter, made = nn.DropoutCounter(seed=7), []

    def segment(x):
        if noise:
            x = x + 0 * torch.rand(3)[0]
        for _ in range(2):
            key = counter.next()
            made.append(key["offset"])
            x = drop(x, key)
        return x

    x = torch.randn(40, 9, requires_grad=True)
    y = x
    for _ in range(3):
        y = checkpoint(segment, y, use_reentrant=reentrant)
    assert made == list(range(6)) and counter.offset == 6
    g, = torch.autograd.grad(y.sum(), x) if not reentrant else (y.sum().backward(), x.grad)[1:]
    assert sorted(made[6:]) == list(range(6)) and counter.offset == 6
    want = torch.ones_like(x)
    for k in range(6):
        want = drop(want, {"seed": 7, "offset": k})
    assert torch.equal(g, want)
    assert counter.next()["offset"] == 6


@pytest.mark.parametrize("outer", [True, False])
@pytest.mark.parametrize("inner", [True, False])
def test_nested_checkpoints(outer, inner):
    counter = nn.DropoutCounter(seed=1)

    def part(x):
        return drop(x, counter.next())

    def whole(x):
        return part(checkpoint(part, part(x), use_reentrant=inner))

    x = torch.randn(30, 5, requires_grad=True)
    checkpoint(whole, x, use_reentrant=outer).sum().backward()
    want = torch.ones_like(x)
    for k in range(3):
        want = drop(want, {"seed": 1, "offset": k})
    assert torch.equal(x.grad, want) and counter.offset == 3


@pytest.mark.parametrize("reentrant", [True, False])
def test_two_forward_passes_before_their_backward_passes(reentrant):
    counter = nn.DropoutCounter(seed=2)
    xs = [torch.randn(30, 5, requires_grad=True) for _ in range(2)]
    ys = [checkpoint(lambda t: drop(t, counter.next()), x, use_reentrant=reentrant) for x in xs]
    for i in (1, 0):
        ys[i].sum().backward()
        assert torch.equal(xs[i].grad, drop(torch.ones(30, 5), {"seed": 2, "offset": i}))


@pytest.mark.parametrize("reentrant", [True, False])
def test_a_recomputation_without_the_generator_state_is_refused(reentrant):
    counter = nn.DropoutCounter(seed=3)
    x = torch.randn(30, 5, requires_grad=True)
    y = checkpoint(lambda t: drop(t, counter.next()), x, use_reentrant=reentrant, preserve_rng_state=False)
    with pytest.raises(RuntimeError, match="recomput"):
        y.sum().backward()
    # with a key from outside it works
    key = counter.next()
    y = checkpoint(lambda t: drop(t, key), x, use_reentrant=reentrant, preserve_rng_state=False)
    x.grad = None
    y.sum().backward()
    assert torch.equal(x.grad, drop(torch.ones(30, 5), key))


@pytest.mark.parametrize("reentrant", [True, False])
def test_the_same_generator_state_gives_the_same_key(reentrant):
    # a program that seeds torch before every forward pass: both recomputations find their masks
    counter, xs, ys = nn.DropoutCounter(seed=4), [], []
    for _ in range(2):
        torch.manual_seed(0)
        xs.append(torch.randn(30, 5, requires_grad=True))
        ys.append(checkpoint(lambda t: drop(t, counter.next()), xs[-1], use_reentrant=reentrant))
    for x, y in zip(xs, ys):
        with torch.no_grad():
            kept = y != 0
        y.sum().backward()
        assert torch.equal(x.grad != 0, kept)


def test_ordinary_calls_leave_the_generator_alone():
    counter = nn.DropoutCounter(seed=5, offset=3)
    before = torch.get_rng_state()
    assert [counter.next()["offset"] for _ in range(3)] == [3, 4, 5]
    assert torch.equal(torch.get_rng_state(), before)
    with torch.no_grad():
        assert [counter.next()["offset"] for _ in range(3)] == [6, 7, 8]
    with torch.inference_mode():
        assert counter.next()["offset"] == 9
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: t):
        assert [counter.next()["offset"] for _ in range(2)] == [10, 11]
    assert counter.state_dict() == {"seed": 5, "offset": 12, "state": None}


def test_remembered_keys_are_bounded():
    counter = nn.DropoutCounter(seed=6)
    with torch.no_grad():
        for _ in range(nn.DropoutCounter._REMEMBERED + 10):
            counter.next()
    assert len(counter._given) == nn.DropoutCounter._REMEMBERED
    # a forward pass longer than that is refused in its backward pass, not given other masks
    x = torch.randn(2, 2, requires_grad=True)
    counter._given.clear()
    y = checkpoint(lambda t: t * counter.next()["offset"], x, use_reentrant=True)
    counter._given.clear()
    with pytest.raises(RuntimeError, match="recomput"):
        y.sum().backward()


def test_threads_get_keys_of_their_own():
    class Slow(int):
        """Lets other threads run between the reading and the writing of the offset."""
        def __add__(self, other):
            time.sleep(0.002)
            return Slow(int(self) + other)

    counter, got = nn.DropoutCounter(seed=8), []
    counter.offset = Slow(0)
    threads = [threading.Thread(target=lambda: got.extend(counter.next()["offset"] for _ in range(5)))
               for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sorted(got) == list(range(20))


def test_copied_modules_share_the_counter_and_not_the_masks():
    counter = nn.DropoutCounter(seed=9)
    block = torch.nn.Sequential(torch.nn.Linear(4, 4), nn.FlashDropout(0.25, counter))
    layers = torch.nn.ModuleList(copy.deepcopy(block) for _ in range(3))
    keys = [layer[1].counter.next()["offset"] for layer in layers] + [block[1].counter.next()["offset"]]
    assert keys == [0, 1, 2, 3]
    assert layers[0][0].weight is not block[0].weight and layers[0][1] is not block[1]
    assert layers[0][1].p == 0.25 and copy.copy(block[1]).counter is counter
    layers[0][1].eval()
    assert block[1].training
    # a counter that is copied by itself is another one
    other = copy.deepcopy(counter)
    other.next()
    assert counter.offset == 4 and other.offset == 5


def test_runs_repeat_from_a_restored_counter_and_generator():
    """The same program twice in one process, from the same state of torch's generator and of the
    counter, in every way to set the latter: same keys, and the counter ends at the same offset."""
    def program(counter):
        with torch.no_grad():
            keys = [counter.next()["offset"] for _ in range(3)]
        x = torch.randn(9, 4, requires_grad=True)
        checkpoint(lambda t: drop(t, counter.next()), x, use_reentrant=False).sum().backward()
        return keys + [counter.next()["offset"], counter.offset]

    counter = nn.DropoutCounter(seed=1)
    saved = counter.state_dict()
    torch.manual_seed(3)
    first = program(counter)
    assert first == [0, 1, 2, 4, 5]
    torch.manual_seed(3)
    counter.offset = 0
    assert program(counter) == first
    torch.manual_seed(3)
    counter.load_state_dict(saved)
    assert program(counter) == first
    # another seed is not answered with keys of the one before
    torch.manual_seed(3)
    counter.load_state_dict({"seed": 2, "offset": 7, "state": None})
    with torch.no_grad():
        assert counter.next() == {"seed": 2, "offset": 7, "state": None}

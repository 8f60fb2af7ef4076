"""Rows sorted by expert on the GPU where the forms end: values that are no
numbers, the form with scratch replayed, on two streams and with a caller's
scratch, and launches that a size cuts in two."""
import numpy as np
import pytest
import torch

import oracle as O
from moe_layer_amd import ops

from gpu_util import dev
from test_gpu_sorted import KINDS, check_sort, routing

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def special_rows(T, cols, seed):
    """bf16 rows whose 128-column groups hold, in turn: numbers, zeros, values under
    the scale's floor, the largest numbers, an infinity, a NaN of either sign and of
    the smallest and the largest bits, both, NaN alone, and negative zeros."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, cols // 128, 128, generator=g).bfloat16()
    bits = x.view(torch.int16)
    for i in range(T * (cols // 128)):
        t, b, at = i // (cols // 128), i % (cols // 128), (37 * i) % 128
        kind = i % 13
        if kind == 1:
            x[t, b] = 0.0
        elif kind == 2:
            x[t, b] *= 2.0 ** -60
        elif kind == 3:
            x[t, b] = torch.where(x[t, b] > 0, 3.3e38, -3.3e38).bfloat16()
        elif kind in (4, 5):
            x[t, b, at] = INF if kind == 4 else -INF
        elif kind in (6, 7, 8, 9):
            bits[t, b, at] = (0x7fc0, 0xffc0 - 0x10000, 0x7f81, 0xffff - 0x10000)[kind - 6]
        elif kind == 10:
            x[t, b, at], x[t, b, (at + 64) % 128] = INF, NAN
        elif kind == 11:
            x[t, b] = NAN
        elif kind == 12:
            x[t, b], x[t, b, at] = -0.0, 2.0 ** -130
    return x.view(T, cols)


@pytest.mark.parametrize("T,k,cols", [
    (1, 8, 7168), (40, 3, 1664),              # every workgroup compares the ids
    (2600, 2, 128), (2600, 3, 512), (1700, 8, 1664), (1100, 4, 20480),   # tokens share a workgroup
    (52000, 1, 128), (26000, 2, 640), (7000, 8, 2048)])                  # counted
def test_sort_to_fp8_is_moe_quant_act_whatever_the_values(T, k, cols):
    """Codes and scales bit for bit, in every form of the sort.  A signaling NaN is
    taken for a quiet one: moe_quant_act's fmaxf of one is a NaN, which drops the
    columns before it from the maximum, so what that makes is a matter of its order."""
    d, E = dev(), 5
    x = special_rows(min(T, 300), cols, T).repeat(-(-T // 300), 1)[:T].contiguous().to(d)
    ids = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(k), dtype=torch.int32).to(d)
    quiet = torch.where(x.isnan(), x.view(torch.int16) | 0x40, x.view(torch.int16)).view(torch.bfloat16)
    codes, scales = ops.moe_quant_act(quiet)
    rows, row_scales, _, inv = ops.moe_sort_rows(x, ids, E, quant="fp8")
    for j in range(k):
        at = inv[:, j].long()
        assert torch.equal(rows[at], codes)
        assert torch.equal(row_scales[at].view(torch.int32), scales.view(torch.int32))


# --------------------------------- few tokens that count, many that compare ---

@pytest.mark.parametrize("kind,quant", KINDS)
@pytest.mark.parametrize("T,k,E,cols", [(32, 64, 100, 256), (33, 64, 1024, 256), (80, 64, 70, 640), (200, 33, 100, 1152),
                                        (255, 64, 64, 128), (256, 16, 300, 512), (49, 64, 65, 17408)])
def test_sort_of_few_tokens_with_many_slots(T, k, E, cols, kind, quant):
    """Both sides of where up to 256 tokens' ids are counted, not compared."""
    rng = np.random.default_rng(T + k)
    check_sort(T, k, E, cols, kind, quant, routing(rng, T, k, E, away=0.1, repeats=k > E), T)


def test_few_tokens_with_many_slots_past_the_last_cache():
    d, T, k, E, cols = dev(), 256, 64, 128, 8192
    g = torch.Generator(device=d).manual_seed(5)
    x = torch.randn(T, cols, generator=g, device=d).bfloat16()
    ids = torch.randint(-2, E + 2, (T, k), generator=g, device=d, dtype=torch.int32)
    rows, _, offsets, inv = ops.moe_sort_rows(x, ids, E)
    assert rows.nbytes >= 256 << 20
    want_off, want_inv, token = O.sort_slots(ids.cpu().numpy(), E)
    np.testing.assert_array_equal(offsets.cpu().numpy(), want_off)
    np.testing.assert_array_equal(inv.cpu().numpy(), want_inv)
    assert torch.equal(rows[:len(token)], x[torch.from_numpy(np.asarray(token)).long().to(d)])


# ------------------------------------------------- the form with scratch ---

COUNTED = dict(T=13001, k=4, E=100, cols=128)             # 52004 slots: counted, placed and moved


def counted_case(seed, T, k, E, cols):
    rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    ids = rng.integers(-3, E + 3, (T, k)).astype(np.int32)
    x = torch.randn(T, cols, generator=g).bfloat16()
    return torch.from_numpy(ids), x, O.sort_slots(ids, E)


def check_counted(x, want, rows, offsets, inv):
    want_off, want_inv, token = want
    np.testing.assert_array_equal(offsets.cpu().numpy(), want_off)
    np.testing.assert_array_equal(inv.cpu().numpy(), want_inv)
    n = int(want_off[-1])
    np.testing.assert_array_equal(rows[:n].view(torch.int16).cpu().numpy(), x.view(torch.int16).numpy()[token])
    assert (rows[n:] == 7).all(), "rows behind the last one were written"


class Buffers:
    """A caller's operands and outputs, and scratch of the size asked for with a guard behind it."""

    def __init__(self, T, k, E, cols):
        d, n = dev(), ops.moe_sort_scratch_bytes(T, k, E)
        assert n > 0
        self.x, self.ids = torch.zeros(T, cols, dtype=torch.bfloat16, device=d), torch.zeros(T, k, dtype=torch.int32, device=d)
        self.rows = torch.empty(T * k, cols, dtype=torch.bfloat16, device=d)
        self.offsets, self.inv = torch.empty(E + 1, dtype=torch.int32, device=d), torch.empty(T, k, dtype=torch.int32, device=d)
        self.room = torch.empty(n + 256, dtype=torch.uint8, device=d)
        self.scratch, self.E = self.room[:n], E

    def fill(self, x, ids):
        self.x.copy_(x)
        self.ids.copy_(ids)
        self.rows.fill_(7)
        self.scratch.fill_(0xff)
        self.room[self.scratch.numel():] = 0xa5

    def sort(self):
        return ops.moe_sort_rows(self.x, self.ids, self.E, rows=self.rows, offsets=self.offsets, inv=self.inv,
                                 scratch=self.scratch)

    def check(self, x, want):
        check_counted(x, want, self.rows, self.offsets, self.inv)
        assert (self.room[self.scratch.numel():] == 0xa5).all(), "wrote behind the scratch"


def test_counted_sort_in_a_callers_scratch():
    """Exactly the bytes asked for, whatever they hold; one byte less is refused."""
    b = Buffers(**COUNTED)
    for seed in (1, 2):
        ids, x, want = counted_case(seed, **COUNTED)
        b.fill(x, ids)
        b.sort()
        b.check(x, want)
    b.scratch = b.scratch[:-1]
    with pytest.raises(ops.MoeError):
        b.sort()


def test_counted_sort_replays():
    """Its three launches from a captured graph: every replay, on other rows and ids
    and with eager work and synchronisation between them, against the definition."""
    b = Buffers(**COUNTED)
    ids, x, want = counted_case(0, **COUNTED)
    b.fill(x, ids)
    b.sort()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.sort()
    other = Buffers(**COUNTED)
    for seed in range(3, 8):
        ids, x, want = counted_case(seed, **COUNTED)
        b.fill(x, ids)
        graph.replay()
        if seed % 2:
            torch.cuda.synchronize()
        other.fill(x, ids)
        other.sort()
        b.check(x, want)
        other.check(x, want)


def test_counted_sort_on_two_streams_of_two_threads():
    """Two threads, a stream, rows and a scratch each, sorting at once."""
    import threading

    sets = [(Buffers(**COUNTED), [counted_case(10 * i + j, **COUNTED) for j in range(4)]) for i in range(2)]
    torch.cuda.synchronize()
    errors = []

    def work(b, cases):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for ids, x, want in cases:
                    b.fill(x, ids)
                    for _ in range(3):
                        b.sort()
                    b.check(x, want)
        except BaseException as e:   # noqa: BLE001 (told to the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=s) for s in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


# -------------------------------------------------- launches cut in two ---

@pytest.mark.parametrize("weighted", [False, True])
def test_combine_of_more_columns_than_a_launch_takes(weighted):
    """T * cols / 8 past 2^31 - 1: the tokens behind that are a launch of their own,
    with their own slots, weights and outputs.  Weights are powers of two and a token
    has one slot, so outputs are exact."""
    d, cols, n = dev(), 8192, 40
    T = (2 ** 31 - 1) // (cols // 8) + 700
    g = torch.Generator(device=d).manual_seed(3)
    rows = torch.randn(n, cols, generator=g, device=d).bfloat16()
    inv = torch.randint(-1, n, (T, 1), generator=g, device=d, dtype=torch.int32)
    w = torch.exp2(torch.randint(-3, 4, (T, 1), generator=g, device=d).float()) if weighted else None
    out = ops.moe_combine_rows(rows, inv, w)
    for lo in range(0, T, 1 << 17):
        part = slice(lo, min(T, lo + (1 << 17)))
        want = torch.where(inv[part] >= 0, rows[inv[part, 0].clamp(min=0).long()].float(), 0.0)
        if weighted:
            want *= w[part]
        assert torch.equal(out[part], want.bfloat16()), lo


# ----------------------------------------------------------- autograd ---

def test_no_output_has_a_grad_fn():
    """Operands that require a gradient are taken, and nothing is recorded: the
    gradients are calls of their own, as the docstrings say."""
    d = dev()
    x = torch.randn(9, 64, device=d).bfloat16().requires_grad_()
    ids = torch.randint(0, 4, (9, 2), device=d, dtype=torch.int32)
    w = torch.rand(9, 2, device=d, requires_grad=True)
    rows, _, _, inv = ops.moe_sort_rows(x, ids, 4)
    out = ops.moe_combine_rows(rows.requires_grad_(), inv, w)
    grads = ops.moe_combine_rows_bwd(out, inv, rows=rows, weights=w)
    for t in (out, *grads):
        assert t.grad_fn is None and not t.requires_grad
    for f in (ops.moe_sort_rows, ops.moe_combine_rows, ops.moe_combine_rows_bwd):
        assert "autograd" in f.__doc__.lower() or "grad_fn" in f.__doc__

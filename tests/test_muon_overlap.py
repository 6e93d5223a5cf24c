"""Which matrices of one update may share memory (no GPU): none that is written
with any other, element by element; column or row slices of one tensor may."""
import random

import pytest
import torch

from linear_cross_entropy_token_gb300.muon import check_muon_tensors


def refused(grads, momenta=None, weights=None, updates=None):
    try:
        check_muon_tensors(grads, momenta, weights, updates)
    except ValueError as e:
        assert "overlaps" in str(e)
        return True
    return False


def z(rows=4, cols=6, dtype=torch.float32):
    return torch.zeros(rows, cols, dtype=dtype)


def test_a_written_matrix_over_another_is_refused():
    big = torch.zeros(64)

    def at(offset, ld=6):
        return big.as_strided((4, 6), (ld, 1), offset)

    g = z()
    assert refused([g], [g])                                      # the momentum in the gradient's place
    assert refused([at(0)], [at(6)])                              # shifted by a row
    assert refused([at(0)], [at(23)])                             # by all but one element
    assert not refused([at(0)], [at(24)])
    assert refused([z(), z()], [at(0), at(5)])                    # two that are written
    assert refused([z(), z()], [at(0, 14), at(5, 14)])            # column slices with one column in common
    assert not refused([z(), z()], [at(0, 14), at(6, 14)])        # without
    assert refused([z(), z()], [at(6, 12), at(1, 12)])
    assert not refused([z(), z()], [at(6, 12), at(0, 12)])
    assert refused([z()], None, [at(0)]) is False
    assert refused([z()], [at(3)], [at(0)])
    w = torch.zeros(4, 6, dtype=torch.bfloat16)
    assert refused([w], None, None, [w])                          # an update over its gradient


def test_gradients_alone_may_share_memory():
    g = z()
    assert not refused([g, g], [z(), z()])
    assert not refused([z(), z()], None, [torch.zeros(4, 12)[:, :6], torch.zeros(4, 12)[:, 6:]])
    fused = torch.zeros(12, 6)
    assert not refused([z() for _ in range(3)], None, list(fused.view(3, 4, 6).unbind(0)))
    fused = torch.zeros(4, 18)
    assert not refused([z() for _ in range(3)], None, list(fused.split(6, 1)))
    # two strides in one tensor, rows that interleave without meeting
    big = torch.zeros(200)
    assert not refused([z()], [big.as_strided((4, 6), (20, 1), 0)], [big.as_strided((4, 6), (40, 1), 8)])
    assert refused([z()], [big.as_strided((4, 6), (20, 1), 0)], [big.as_strided((4, 6), (40, 1), 4)])


@pytest.mark.parametrize("seed", range(20))
def test_against_the_elements_themselves(seed):
    """Random slices of one buffer, of one or two strides and types: refused just where an element is shared."""
    rng = random.Random(seed)
    buffer = torch.zeros(600, dtype=torch.uint8)
    for _ in range(200):
        rows, cols = rng.randint(1, 6), rng.randint(1, 5)

        def view(dtype):
            es = dtype.itemsize
            ld = rng.choice((cols, cols + 1, 2 * cols, rng.randint(cols, 12)))
            need = ((rows - 1) * ld + cols) * es
            at = rng.randrange(0, (600 - need) // 4 + 1) * 4
            t = buffer[at:at + need].view(dtype).as_strided((rows, cols), (ld, 1))
            touched = {at + (r * ld + c) * es + b for r in range(rows) for c in range(cols) for b in range(es)}
            return t, touched

        types = rng.choice(((torch.float32, torch.float32), (torch.bfloat16, torch.float32)))
        g, gs = view(types[0])
        m, ms = view(torch.float32)
        w, ws = view(types[1])
        shared = bool(gs & ms or gs & ws or ms & ws)
        assert refused([g], [m], [w]) == shared, (g.stride(), m.stride(), w.stride())

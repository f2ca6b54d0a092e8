"""The handle of an int8 weight: what it tells the kernels has to be what its planes hold now."""
import copy
import pickle

import numpy as np
import pytest
import torch

import bit_rotated_weight_b200 as tq

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


class Plane:
    """A stand-in for a CUDA tensor, for checks of the handle without a GPU."""
    is_cuda, device = True, torch.device("cuda:0")

    def __init__(self, shape, dtype, at, offset=0):
        self.shape, self.dtype, self.at, self.offset = torch.Size(shape), dtype, at, offset
        self.held = (self.shape.numel() + offset) * dtype.itemsize

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.device.index

    def storage_offset(self):
        return self.offset

    def data_ptr(self):
        return self.at + self.offset * self.dtype.itemsize

    def untyped_storage(self):
        return self

    def nbytes(self):
        return self.held


def planes(E=2, n=8, k=32, offset=0):
    return Plane((E, n, k), torch.int8, 4096, offset), Plane((E, n), torch.float32, 65536)


def test_handle_follows_planes_that_move():
    q, s = planes()
    w = tq.Int8Weight(q, s, 8, 32, 2)
    st = w.c_struct()
    assert (st.q, st.wscale) == (4096, 65536) and w.c_struct() is st
    q.at = 8192
    assert (w.c_struct().q, w.c_struct().wscale) == (8192, 65536)
    s.at = 1 << 20
    assert (w.c_struct().q, w.c_struct().wscale) == (8192, 1 << 20)
    q.at, q.device = 16384, torch.device("cuda:1")
    with pytest.raises(ValueError, match="one CUDA device"):
        w.c_struct()


def test_handle_refuses_planes_whose_storage_is_gone():
    # (a slice of a larger storage has an address that is not 0 even then)
    q, s = planes(offset=64)
    w = tq.Int8Weight(q, s, 8, 32, 2)
    w.c_struct()
    q.at = q.held = 0
    with pytest.raises(ValueError, match="storage"):
        w.c_struct()
    q.at, q.held = 32768, 64 + 2 * 8 * 32
    assert w.c_struct().q == 32768 + 64


def test_handle_takes_planes_of_its_shape_only():
    E, n, k = 2, 8, 32

    def handle(qs, ss):
        return tq.Int8Weight(Plane(qs, torch.int8, 4096), Plane(ss, torch.float32, 65536), n, k, E).c_struct()

    for qs in ((E, n, k), (E * n, k), (E * n * k,)):
        for ss in ((E, n), (E * n,), (E, n, 1), (E * n, 1)):
            assert handle(qs, ss).q == 4096
    for qs in ((E, k, n), (k, E * n), (n, E, k), (1, E * n, k), (E, n, k, 1), (E, n, k - 1), (E * k, n)):
        with pytest.raises(ValueError, match="Int8Weight.q"):
            handle(qs, (E, n))
    for ss in ((n, E), (1, E * n), (E, 1, n), (E, n + 1)):
        with pytest.raises(ValueError, match="Int8Weight.wscale"):
            handle((E, n, k), ss)
    one = tq.Int8Weight(Plane((n, k), torch.int8, 4096), Plane((n,), torch.float32, 65536), n, k, 1)
    assert one.c_struct().n == n
    with pytest.raises(ValueError, match="Int8Weight.q"):
        tq.Int8Weight(Plane((k, n), torch.int8, 4096), Plane((n,), torch.float32, 65536), n, k, 1).c_struct()


def test_a_handle_that_was_used_can_be_copied_and_pickled():
    q, s = planes()
    w = tq.Int8Weight(q, s, 8, 32, 2)
    w.c_struct()
    shared, own, loaded = copy.copy(w), copy.deepcopy(w), pickle.loads(pickle.dumps(w))
    assert shared.q is q and own.q is not q and loaded.q is not q
    for v in (shared, own, loaded):
        assert (v.n, v.k, v.num_experts, v.nbytes) == (8, 32, 2, w.nbytes)
    own.q.at, loaded.wscale.at = 8192, 1 << 20             # (planes of their own, elsewhere)
    assert (own.c_struct().q, loaded.c_struct().wscale) == (8192, 1 << 20)
    assert (w.c_struct().q, w.c_struct().wscale) == (4096, 65536)


# ------------------------------------------------------------------ on the GPU
def small(seed, E=1, n=64, k=96):
    return tq.tq4_1s_int8_quantize(torch.randn(E, n, k, generator=torch.Generator().manual_seed(seed)).to(DEV))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 40])
def test_calls_read_the_storage_that_the_planes_have_now(m):
    x = torch.randn(m, 96, generator=torch.Generator().manual_seed(m)).to(DEV)
    for made in (lambda v: v, lambda v: tq.Int8Weight(v.q.clone(), v.wscale.clone(), 64, 96, 1)):
        w, other = made(small(1)), small(2)
        want, first = tq.tq4_1s_linear_int8(x, other), tq.tq4_1s_linear_int8(x, w)
        assert not torch.equal(first, want)
        old = w.q.detach(), w.wscale.detach()             # (both storages live on)
        w.q.set_(other.q.untyped_storage(), 0, other.q.shape, other.q.stride())
        w.wscale.data = other.wscale
        assert torch.equal(tq.tq4_1s_linear_int8(x, w), want)
        assert torch.equal(tq.tq4_1s_int8_dequantize(w), tq.tq4_1s_int8_dequantize(other))
        w.q.data, w.wscale.data = old
        assert torch.equal(tq.tq4_1s_linear_int8(x, w), first)


@pytest.mark.gpu
def test_experts_moved_out_and_back():
    # the codes leave the card and come back to another place
    up, down = small(3, 4, 64, 96), small(4, 4, 96, 64)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(20, 96, generator=g).to(torch.bfloat16).to(DEV)
    ids = torch.randint(0, 4, (20, 2), generator=g, dtype=torch.int32).to(DEV)
    tw = torch.rand(20, 2, generator=g).to(DEV)
    want = tq.tq4_1s_moe_int8(x, ids, tw, up, down)
    host, storage = up.q.cpu(), up.q.untyped_storage()
    size = storage.nbytes()
    torch.cuda.synchronize()
    storage.resize_(0)
    with pytest.raises(ValueError, match="storage"):
        tq.tq4_1s_moe_int8(x, ids, tw, up, down)
    with pytest.raises(ValueError, match="storage"):
        tq.tq4_1s_int8_dequantize(up)
    taken = torch.full((size,), 7, dtype=torch.uint8, device=DEV)      # (where the codes were, perhaps)
    storage.resize_(size)
    up.q.copy_(host)
    assert torch.equal(tq.tq4_1s_moe_int8(x, ids, tw, up, down), want)
    assert bool((taken == 7).all())
    assert np.array_equal(up.q.cpu().numpy(), host.numpy())


@pytest.mark.gpu
def test_a_transposed_plane_is_refused():
    w = small(6)
    x = torch.ones(3, 96, device=DEV)
    want = tq.tq4_1s_linear_int8(x, w)
    turned = tq.Int8Weight(w.q[0].t().contiguous(), w.wscale, 64, 96, 1)
    with pytest.raises(ValueError, match="Int8Weight.q"):
        tq.tq4_1s_linear_int8(x, turned)
    assert torch.equal(tq.tq4_1s_linear_int8(x, tq.Int8Weight(w.q[0], w.wscale[0], 64, 96, 1)), want)


@pytest.mark.gpu
def test_copies_of_a_used_handle_multiply_alike():
    w, x = small(7), torch.ones(3, 96, device=DEV)
    want = tq.tq4_1s_linear_int8(x, w)
    own, loaded = copy.deepcopy(w), pickle.loads(pickle.dumps(w))
    w.q.zero_()
    for v in (own, loaded):
        assert torch.equal(tq.tq4_1s_linear_int8(x, v), want)

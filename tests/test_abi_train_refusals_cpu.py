"""Refusals of the calls of include/usaf_train.h and of their binding that keep bad pointers off the
GPU, checked on the host."""
import ctypes

import pytest
import torch

from sparse_moe_fine_gb300 import binding as B

fake_addresses = pytest.mark.skipif(torch.cuda.is_available(),
                                    reason="fake device addresses; run where no GPU is visible")
FAKE = ctypes.c_void_p(4096)  # never dereferenced: the calls below fail on the host


@fake_addresses
@pytest.mark.parametrize("at", [4097, 4098, 4100, 4104])
def test_aux_workspace_has_to_be_aligned(at):
    """fp32 and int32 partial sums are stored from the workspace's start on."""
    r = B.lib().usaf_router_aux_fwd(8, 4, 2, FAKE, 4, FAKE, None, None, 1, 1.0, 1.0, FAKE, FAKE, FAKE,
                                    FAKE, None, ctypes.c_void_p(at), 1 << 30, None)
    assert r == 1


def test_routing_tables_may_be_absent_or_addresses():
    """A routing whose fields are None or bare addresses reaches the library, which refuses what it
    needs and does not have."""
    t = torch.zeros(4, dtype=torch.int32)
    r = B.Routing(t, None, 4096, t, None, 0, t).c()
    got = [getattr(r, f) for f, _ in B._Routing._fields_]
    assert got[0] == got[3] == got[6] == t.data_ptr() and got[2] == 4096
    assert got[1] is None and got[4] is None and not got[5]
    s = B.shape(4, 64, 4, 2, 64)
    with pytest.raises(B.UsafError):
        B.route_topk_noalloc(s, None, None, B.Routing(*[None] * 7), logits_in=4096, stream=0)


class _Tensor:
    """What the binding reads of a CUDA tensor, without one."""

    def __init__(self, shape, dtype=torch.float32, dev=0, at=1 << 20, contiguous=True):
        self.shape, self.dtype, self.dev, self.at = torch.Size(shape), dtype, dev, at
        self.contiguous = contiguous
        self.device = torch.device("cuda", dev) if dev >= 0 else torch.device("cpu")

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return self.contiguous

    def stride(self):
        st = [1]
        for n in reversed(self.shape[1:]):
            st.insert(0, st[0] * n)
        return tuple(st)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    @property
    def nbytes(self):
        return self.numel() * self.dtype.itemsize

    def data_ptr(self):
        return self.at


class _Lib:
    """Records the calls that reach the library."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if "size" in name or "capacity" in name:
            return getattr(self.real, name)
        return lambda *a: self.calls.append((name, a)) or 0


S = B.shape(8, 64, 4, 2, 64)
I32, U8, I8, BF = torch.int32, torch.uint8, torch.int8, torch.bfloat16


def _calls(d=0, d2=None, ws=None, status=None, rt=None):
    """The four calls with all tensors on device d, the last one on d2."""
    T = lambda *a, **k: _Tensor(*a, dev=d, **k)
    d2 = d if d2 is None else d2
    cap = B.routed_rows_capacity(S)
    store = lambda: B.ActStore8(*[T(sh, dt) for sh, dt in zip(B.ActStore8.shapes(S),
                                                              (I8, U8, I8, U8))])
    rt = rt or _routing(d)
    w = ws or T((1 << 20,), U8)
    return dict(
        fwd=lambda st=None: B.router_aux_fwd(
            T((8, 4)), T((16,), I32), 2, T((1, 4), I32), T((1, 4)), T((1,), I32),
            _Tensor((3,), dev=d2), 1.0, 1.0, ws=w, dev_status=status, stream=st),
        bwd=lambda st=None: B.router_aux_bwd(
            T((8, 4)), 2, T((1, 4), I32), T((1,), I32), _Tensor((8, 4), dev=d2), 1.0, 1.0,
            dev_status=status, stream=st),
        grad=lambda st=None: B.router_grad(
            T((8, 4)), T((8, 64), BF), T((4, 64)), g_router=T((4, 64)),
            dx=_Tensor((8, 64), BF, dev=d2), ws=w, dev_status=status, stream=st),
        save=lambda st=None: B.act8_save(S, T((8, 64), BF), _Tensor((128, cap), BF, dev=d2), rt,
                                         store(), dev_status=status, stream=st),
        restore=lambda st=None: B.act8_restore(S, store(), rt, T((64, cap), BF), T((128, cap), BF),
                                               _Tensor((64, cap), BF, dev=d2), stream=st))


def _routing(d, **other):
    cap = B.routed_rows_capacity(S)
    f = dict(topk_idx=(16,), topk_w=(16,), expert_count=(4,), expert_offset=(5,), perm_tok=(cap,),
             perm_slot=(cap,), slot_row=(16,))
    f = {n: _Tensor(sh, torch.float32 if n == "topk_w" else I32, dev=d) for n, sh in f.items()}
    return B.Routing(**{**f, **other})


NAMES = ["fwd", "bwd", "grad", "save", "restore"]


@pytest.fixture
def fake(monkeypatch):
    lib = _Lib(B.lib())
    monkeypatch.setattr(B, "lib", lambda: lib)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return lib


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device_are_refused(fake, name):
    _calls()[name]()
    assert len(fake.calls) == 1
    for call in (_calls(d2=1)[name], _calls(d=1)[name], _calls(d=-1)[name]):
        with pytest.raises(ValueError):
            call()
    assert len(fake.calls) == 1


@pytest.mark.parametrize("name", ["fwd", "grad"])
def test_workspaces_off_the_device_or_strided_are_refused(fake, name):
    for bad in (_Tensor((1 << 20,), U8, dev=-1), _Tensor((1 << 20,), U8, dev=1),
                _Tensor((1 << 20,), U8, contiguous=False)):
        with pytest.raises(ValueError):
            _calls(ws=bad)[name]()
    assert not fake.calls
    _calls(ws=_Tensor((1 << 18,), I32))[name]()  # its size in bytes counts
    a = fake.calls[0][1]
    assert a[-2] == 1 << 20


@pytest.mark.parametrize("name", ["fwd", "bwd", "grad", "save"])
def test_status_words_off_the_device_or_too_small_are_refused(fake, name):
    for bad in (_Tensor((1,), I32, dev=-1), _Tensor((1,), I32, dev=1), _Tensor((0,), I32),
                _Tensor((1,), U8)):
        with pytest.raises(ValueError):
            _calls(status=bad)[name]()
    assert not fake.calls
    _calls(status=_Tensor((1,), I32))[name]()
    _calls(status=4096)[name]()  # an address
    assert len(fake.calls) == 2


@pytest.mark.parametrize("name,fields", [("save", ["expert_offset"]),
                                         ("restore", ["topk_w", "expert_offset", "perm_tok",
                                                      "perm_slot"])])
def test_routing_tables_of_another_shape_are_refused(fake, name, fields):
    """Rows are addressed by them: a routing of another shape would be read and written past the ends."""
    for f in fields:
        n = getattr(_routing(0), f).numel()
        dt = torch.float32 if f == "topk_w" else I32
        for bad in (_Tensor((n - 1,), dt), _Tensor((n,), torch.int64), _Tensor((n,), dt, dev=-1),
                    _Tensor((n,), dt, contiguous=False)):
            with pytest.raises(ValueError):
                _calls(rt=_routing(0, **{f: bad}))[name]()
    assert not fake.calls
    _calls(rt=_routing(0, **{f: 4096 for f in fields}))[name]()  # addresses
    assert len(fake.calls) == 1

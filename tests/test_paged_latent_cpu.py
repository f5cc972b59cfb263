"""CPU tests of the paged append and latent attention calls' boundary (no kernel runs here): every
refusal of the host checks, the calls that have nothing to do, views that must not be refused, and
what the Python functions refuse before the C call."""
import ctypes

import pytest
import torch

import rope_partial_inplace_amd as ra

OK, NULLPTR, INVALID, RUNTIME = 0, ra.ROPE_ERR_PARAM_NULLPTR, ra.ROPE_ERR_PARAM_INVALID, ra.ROPE_ERR_RUNTIME
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
CODES = {F32: 0, F16: 1, BF16: 2, torch.int64: 3}
HAS_GPU = torch.cuda.is_available()  # there a valid call would launch on these host buffers


def desc(t, **override):
    """A rope_tensor of a host tensor (refusals come before any access); None stays NULL."""
    if t is None:
        return None
    d = ra.RopeTensor()
    d.data = override.get("data", t.data_ptr() if t.numel() else None)
    d.dtype = override.get("dtype", CODES.get(t.dtype, 9))
    d.ndim = override.get("ndim", t.dim())
    shape, stride = override.get("shape", t.shape), override.get("stride", t.stride())
    for i in range(min(4, len(shape))):
        d.shape[i], d.stride[i] = shape[i], stride[i]
    return d


def ref(d):
    return None if d is None else ctypes.byref(d)


def zeros(*shape, dtype=BF16):
    """Zeros on a 16-byte boundary."""
    return torch.zeros(shape, dtype=dtype)


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int64)


class Call:
    """Arguments of one C call by name: tensors, descriptions or plain values."""
    fn, names, tensors, options = None, (), {}, {}

    def __init__(self):
        self.args = {**self.tensors(), **self.plain()}

    def run(self, **change):
        a = {**self.args, **change}
        values = []
        self.keep = []
        for n in self.names:
            v = a[n]
            if isinstance(v, torch.Tensor):
                v = desc(v)
            self.keep.append(v)
            values.append(ref(v) if isinstance(v, ra.RopeTensor) else v)
        st = getattr(ra.LIB, self.fn)(*values)
        assert (st == OK) == (ra.last_error() == "")
        return st

    def changed(self, name, **override):
        """The call with the description of one tensor changed."""
        return self.run(**{name: desc(self.args[name], **override)})


class Append(Call):
    fn = "rope_append_paged_cache"
    names = ("positions", "slots", "query", "key", "value", "table", "q_start", "k_start", "neox",
             "query_out", "key_cache", "value_cache", "stream")

    def tensors(self):
        return dict(positions=ints(5), slots=ints(5), query=zeros(5, 4, 96), key=zeros(5, 2, 128),
                    value=zeros(5, 2, 64), table=zeros(50, 64), query_out=zeros(5, 4, 96),
                    key_cache=zeros(3, 16, 2, 128), value_cache=zeros(3, 16, 2, 64))

    def plain(self):
        return dict(q_start=32, k_start=64, neox=1, stream=None)


class Paged(Call):
    fn = "rope_latent_attention_paged"
    names = ("query", "cache", "page_table", "seq_lens", "query_offsets", "latent", "scale", "out",
             "lse", "workspace", "workspace_bytes", "stream")

    def tensors(self):
        need = ra.LIB.rope_latent_attention_paged_workspace(6, 4, 128, 3)
        self.memory = torch.zeros(need + 64, dtype=torch.uint8)
        return dict(query=zeros(6, 4, 192), cache=zeros(8, 16, 192), page_table=ints(3, 4),
                    seq_lens=ints(3), query_offsets=ints(4), out=zeros(6, 4, 128),
                    lse=zeros(6, 4, dtype=F32))

    def plain(self):
        return dict(latent=128, scale=0.1, workspace=self.memory.data_ptr(),
                    workspace_bytes=self.memory.numel(), stream=None)


class Forward(Call):
    fn = "rope_latent_attention"
    names = ("query", "key", "key_rope", "value", "query_offsets", "key_offsets", "num", "scale",
             "causal", "out", "lse", "stream")

    def tensors(self):
        return dict(query=zeros(6, 2, 128), key=zeros(9, 2, 64), key_rope=zeros(9, 64),
                    value=zeros(9, 2, 64), query_offsets=ints(4), key_offsets=ints(4),
                    out=zeros(6, 2, 64), lse=zeros(6, 2, dtype=F32))

    def plain(self):
        return dict(num=0, scale=0.1, causal=1, stream=None)


class Backward(Forward):
    fn = "rope_latent_attention_backward"
    names = (("grad",) + Forward.names[:4] + ("out", "lse") + Forward.names[4:9] +
             ("dquery", "dkey", "dkey_rope", "dvalue", "workspace", "workspace_bytes", "stream"))

    def tensors(self):
        t = super().tensors()
        need = ra.LIB.rope_latent_attention_backward_workspace(6, 9, 2)
        self.memory = torch.zeros(need + 64, dtype=torch.uint8)
        return dict(t, grad=zeros(6, 2, 64), dquery=zeros(6, 2, 128), dkey=zeros(9, 2, 64),
                    dkey_rope=zeros(9, 64), dvalue=zeros(9, 2, 64))

    def plain(self):
        return dict(super().plain(), workspace=self.memory.data_ptr(),
                    workspace_bytes=self.memory.numel())


CALLS = {"append": Append, "paged": Paged, "forward": Forward, "backward": Backward}
OUTPUTS = {"append": ("query_out", "key_cache", "value_cache"), "paged": ("out", "lse"),
           "forward": ("out", "lse"), "backward": ("dquery", "dkey", "dkey_rope", "dvalue")}
OPTIONAL = {"append": set(), "paged": {"query_offsets", "lse"}, "forward": set(), "backward": set()}
TENSORS = [(c, n) for c in CALLS for n in CALLS[c]().tensors()]


@pytest.mark.skipif(HAS_GPU, reason="reaches the launch, with host buffers")
@pytest.mark.parametrize("call", CALLS)
def test_valid_calls_reach_the_launch(call):
    assert CALLS[call]().run() == RUNTIME


@pytest.mark.parametrize("call,name", TENSORS)
def test_every_tensor_is_checked(call, name):
    c = CALLS[call]()
    t = c.args[name]
    if name not in OPTIONAL[call]:
        assert c.run(**{name: None}) == NULLPTR
    assert c.changed(name, data=None) == NULLPTR
    for ndim in (0, 5, -1, t.dim() + 1 if t.dim() < 4 else 3):
        assert c.changed(name, ndim=ndim, shape=(*t.shape, 1),
                         stride=(*t.stride(), 1)) in (INVALID, NULLPTR)
    for dtype in (-1, 4, 9, 0 if t.dtype != F32 else 1, 3 if t.dtype != torch.int64 else 0):
        assert c.changed(name, dtype=dtype) == INVALID
    for d in range(t.dim()):  # one more, and a negative number of elements, in each dimension
        # (more cached pages, page rows and table rows are as good)
        free = {"append": {"table": (0,), "key_cache": (), "value_cache": ()},
                "paged": {"cache": (0, 1), "page_table": (1,)}}.get(call, {}).get(name, ())
        if d not in free:
            shape = list(t.shape)
            shape[d] += 1
            assert c.changed(name, shape=shape) == INVALID, (d, shape)
        shape = list(t.shape)
        shape[d] = -1
        assert c.changed(name, shape=shape) == INVALID
        stride = list(t.stride())
        stride[d] = -stride[d]
        assert c.changed(name, stride=stride) == INVALID
        stride[d] = 1 << 62
        assert c.changed(name, stride=stride) == INVALID
    if t.is_floating_point() and t.dim() > 1:
        stride = [2 * s for s in t.stride()]
        assert c.changed(name, stride=stride) == INVALID  # no unit inner stride


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in OUTPUTS[c]])
def test_outputs_overlap_nothing(call, name):
    c = CALLS[call]()
    out = c.args[name]
    for other, t in c.args.items():
        if not isinstance(t, torch.Tensor) or other == name:
            continue
        if call == "append" and (name, other) == ("query_out", "query"):
            continue  # may be the same view; see below
        first = t.data_ptr()
        last = first + (t.numel() - 1) * t.element_size() // 16 * 16
        assert c.changed(name, data=first) == INVALID, other
        assert c.changed(name, data=last // 16 * 16) == INVALID, other
    if "workspace" in c.args:
        assert c.changed(name, data=c.args["workspace"]) == INVALID
    if call != "append":  # outputs are contiguous and aligned there
        shape, stride = list(out.shape), list(out.stride())
        stride[0] += 8
        assert c.changed(name, stride=stride) == INVALID
        if out.dtype != F32:
            assert c.changed(name, data=out.data_ptr() + 2) == INVALID
    else:
        stride = list(out.stride())
        stride[1] = 0
        assert c.changed(name, stride=stride) == INVALID  # reaches elements twice


@pytest.mark.parametrize("call", ["paged", "forward", "backward"])
@pytest.mark.parametrize("name", ["query", "key", "key_rope", "value", "cache", "grad"])
def test_rows_of_attention_inputs_are_aligned(call, name):
    c = CALLS[call]()
    t = c.args.get(name)
    if t is None:
        return
    assert c.changed(name, data=t.data_ptr() + 2) == INVALID
    stride = list(t.stride())
    stride[0] += 4
    assert c.changed(name, stride=stride) == INVALID
    if call != "paged":  # tokens 32 MiB apart
        stride[0] = 1 << 24
        assert c.changed(name, stride=stride) == INVALID


@pytest.mark.parametrize("call", ["paged", "forward", "backward"])
def test_scales_are_finite(call):
    for scale in (float("nan"), float("inf"), -float("inf")):
        assert CALLS[call]().run(scale=scale) == INVALID


@pytest.mark.parametrize("call", ["paged", "backward"])
def test_workspaces(call):
    c = CALLS[call]()
    need = c.args["workspace_bytes"] - 64
    assert c.run(workspace=None) == NULLPTR
    assert c.run(workspace_bytes=need - 1) == INVALID
    assert c.run(workspace_bytes=0) == INVALID
    assert c.run(workspace_bytes=-1) == INVALID
    assert c.run(workspace=c.args["workspace"] + 8) == INVALID
    for t in c.args.values():
        if isinstance(t, torch.Tensor):
            for at in (t.data_ptr(), t.data_ptr() - need):
                at = at // 16 * 16 + (16 if at < t.data_ptr() else 0)
                assert c.run(workspace=at) == INVALID


def test_workspace_sizes():
    paged, back = (ra.LIB.rope_latent_attention_paged_workspace,
                   ra.LIB.rope_latent_attention_backward_workspace)
    for args in ((0, 4, 128, 1), (1, 0, 128, 1), (1, 4, 128, 0), (-5, 4, 128, 1), (1, 4, -1, 1)):
        assert paged(*args) == 0
    assert back(0, 0, 4) == 0 and back(-1, 3, 4) == 0 and back(3, 5, 0) == 0
    assert back(3, 5, 4) >= (3 * 4 + 5 * 4 * 64) * 4
    big = 2 ** 62  # what the calls refuse needs none
    assert paged(big, 4, 512, 1) == paged(4, big, 512, 1) == paged(4, 4, big, 1) == 0
    assert paged(4, 4, 512, big) == paged(4, 4, 512, 2 ** 63 - 1) > 0
    assert back(big, 4, 4) == back(4, big, 4) == back(4, 4, big) == back(2 ** 29, 4, 2 ** 29) == 0
    assert paged(1, 1, 512, 1) <= paged(1, 64, 512, 1) == paged(10 ** 6, 128, 512, 3)


def test_append_options():
    c = Append()
    for name, other in (("query", "query_out"), ("value", "value_cache")):
        assert c.run(**{name: None}) == NULLPTR and c.run(**{other: None}) == NULLPTR
    for start in (-1, 33, 1 << 62):
        assert c.run(q_start=start) == INVALID
    for start in (-1, 65, -(1 << 62)):
        assert c.run(k_start=start) == INVALID
    assert c.run(table=zeros(0, 64)) == INVALID
    assert c.run(table=zeros(50, 0)) == INVALID
    assert c.run(table=zeros(50, 63)) == INVALID  # odd
    assert c.run(table=zeros(50, 98)) == INVALID  # wider than a query head
    assert c.run(value_cache=zeros(4, 16, 2, 64)) == INVALID
    assert c.run(value_cache=zeros(3, 8, 2, 64)) == INVALID
    q = c.args["query"]
    # in place: the same view only
    assert c.run(query_out=desc(q, data=q.data_ptr() + 16)) == INVALID
    assert c.run(query_out=desc(q, stride=(384, 192, 1))) == INVALID
    wide = (1 << 12, 1 << 13)  # 2^25 elements a token
    big = desc(q, shape=(5, *wide), stride=(1 << 25, 1 << 13, 1))
    far = desc(q, data=q.data_ptr() + (1 << 40), shape=(5, *wide), stride=(1 << 25, 1 << 13, 1))
    assert c.run(query=big, query_out=far) == INVALID


def test_paged_options():
    c = Paged()
    for latent in (0, -128, 64, 127, 384, 1024):
        assert c.run(latent=latent) == INVALID
    assert c.run(latent=256) == INVALID  # rows of another width
    assert c.run(query_offsets=ints(3)) == INVALID
    assert c.run(query_offsets=None, seq_lens=ints(4), page_table=ints(4, 4)) == INVALID  # 6 % 4
    assert c.run(query_offsets=None, seq_lens=ints(0), page_table=ints(0, 4)) == INVALID
    huge = 1 << 30
    t = c.args["page_table"]
    assert c.changed("page_table", shape=(3, huge), stride=(0, 0)) == INVALID
    assert c.changed("page_table", shape=(3, huge // 16), stride=(0, 0)) == INVALID
    assert c.changed("cache", shape=(huge, 16, 192), stride=(0, 192, 1)) == INVALID
    assert t is c.args["page_table"]


def test_expanded_options():
    for call in (Forward, Backward):
        c = call()
        assert c.run(query_offsets=None) == NULLPTR and c.run(key_offsets=None) == NULLPTR
        assert c.run(key_offsets=ints(5)) == INVALID
        assert c.run(num=2) == INVALID
        assert c.run(query_offsets=ints(0), key_offsets=ints(0)) == INVALID
        none = dict(query_offsets=None, key_offsets=None)
        for num in (0, -1, 2, 6):  # of 6 queries and 9 keys
            assert c.run(num=num, **none) == INVALID
        assert c.run(key=zeros(9, 2, 96), value=zeros(9, 2, 96)) == INVALID
        assert c.run(key_rope=zeros(9, 32)) == INVALID
        assert c.run(value=zeros(9, 2, 128)) == INVALID


def test_calls_without_work_launch_nothing():
    c = Append()
    empty = dict(positions=ints(0), slots=ints(0), query=zeros(0, 4, 96), key=zeros(0, 2, 128),
                 value=zeros(0, 2, 64), query_out=zeros(0, 4, 96))
    assert c.run(**empty) == OK
    assert c.run(key=zeros(5, 0, 128), key_cache=zeros(3, 16, 0, 128), value=None,
                 value_cache=None, query=None, query_out=None) == OK
    assert c.run(key_cache=zeros(0, 16, 2, 128), value_cache=zeros(0, 16, 2, 64), query=None,
                 query_out=None) == OK  # a cache without pages takes nothing
    c = Paged()
    assert c.run(query=zeros(0, 4, 192), out=zeros(0, 4, 128), lse=zeros(0, 4, dtype=F32)) == OK
    assert c.run(query=zeros(6, 0, 192), out=zeros(6, 0, 128), lse=zeros(6, 0, dtype=F32),
                 workspace=None, workspace_bytes=0) == OK
    assert c.run(query_offsets=ints(1), seq_lens=ints(0), page_table=ints(0, 4), workspace=None,
                 workspace_bytes=0) == OK
    c = Forward()
    no_queries = dict(query=zeros(0, 2, 128), out=zeros(0, 2, 64), lse=zeros(0, 2, dtype=F32))
    assert c.run(**no_queries) == OK
    assert c.run(query_offsets=ints(1), key_offsets=ints(1)) == OK
    c = Backward()
    assert c.run(**no_queries, grad=zeros(0, 2, 64), dquery=zeros(0, 2, 128), key=zeros(0, 2, 64),
                 key_rope=zeros(0, 64), value=zeros(0, 2, 64), dkey=zeros(0, 2, 64),
                 dkey_rope=zeros(0, 64), dvalue=zeros(0, 2, 64), workspace=None,
                 workspace_bytes=0) == OK


@pytest.mark.skipif(HAS_GPU, reason="reaches the launch, with host buffers")
def test_views_that_share_memory_without_overlap_are_accepted():
    c = Append()
    qkv = zeros(5, 8, 160)  # columns of one projection
    assert c.run(query=qkv[:, :4, :96], key=qkv[:, 4:6, :128], value=qkv[:, 6:, :64]) == RUNTIME
    both = zeros(3, 16, 2, 192)  # keys and values of a row side by side
    assert c.run(key_cache=both[..., :128], value_cache=both[..., 128:]) == RUNTIME
    both = zeros(3, 2, 16, 192)  # heads before rows
    assert c.run(key_cache=both[..., :128].transpose(1, 2),
                 value_cache=both[..., 128:].transpose(1, 2)) == RUNTIME
    both = zeros(3, 2, 16, 2, 128)  # keys and values of a page in turn
    assert c.run(key_cache=both[:, 0], value_cache=both[:, 1, ..., :64]) == RUNTIME
    assert c.run(key_cache=both[:, 0], value_cache=both[:, 0, ..., :64]) == INVALID
    assert c.run(query_out=c.args["query"]) == RUNTIME  # in place
    assert c.run(query=None, query_out=None) == RUNTIME
    assert c.run(value=None, value_cache=None) == RUNTIME
    q = c.args["query"]
    assert c.run(query=desc(q, stride=(0, 96, 1))) == RUNTIME  # one query broadcast
    c = Paged()
    wide = zeros(8, 16, 256)
    assert c.run(cache=wide[..., :192], lse=None) == RUNTIME
    assert c.run(query_offsets=None) == RUNTIME
    assert c.run(scale=0.0) == RUNTIME and c.run(scale=-1.0) == RUNTIME
    c = Forward()
    kv = zeros(9, 2, 128)
    assert c.run(key=kv[..., :64], value=kv[..., 64:]) == RUNTIME
    assert c.run(num=3) == RUNTIME
    assert c.run(num=3, query_offsets=None, key_offsets=None) == RUNTIME
    c = Backward()
    assert c.run(key=kv[..., :64], value=kv[..., 64:], grad=zeros(6, 2, 128)[..., :64]) == RUNTIME


def python_calls():
    a, p, f, b = Append().args, Paged().args, Forward().args, Backward().args
    yield lambda: ra.rope_append_paged_cache(a["positions"], a["slots"], a["key"], a["key_cache"],
                                             a["table"], a["value"], a["value_cache"])
    yield lambda: ra.rope_latent_attention_paged(p["query"], p["cache"], p["page_table"],
                                                 p["seq_lens"], 128, 0.1)
    yield lambda: ra.rope_latent_attention(f["query"], f["key"], f["key_rope"], f["value"], 0.1)
    yield lambda: ra.rope_latent_attention_backward(b["grad"], b["query"], b["key"], b["key_rope"],
                                                    b["value"], b["out"], b["lse"], 0.1)
    yield lambda: ra.latent_attention(f["query"], f["key"], f["key_rope"], f["value"], 0.1)


@pytest.mark.parametrize("n", range(5))
def test_python_functions_refuse_host_tensors(n):
    with pytest.raises(ra.RopeError) as e:
        list(python_calls())[n]()
    assert e.value.code == INVALID and "GPU memory" in str(e.value)


def test_python_functions_refuse_mixed_devices():
    """Checked with stand-ins: what counts is the device number of tensors that hold elements."""
    class On:
        def __init__(self, dev, n=1):
            self.dev, self.n = dev, n

        def get_device(self):
            return self.dev

        def numel(self):
            return self.n

    where = ra._device_index
    assert where([On(1), None, On(1)]) == 1
    assert where([On(-1, 0), On(0), On(1, 0)]) == 0
    assert where([On(-1, 0)]) == where([]) == -1
    for bad in ([On(-1)], [On(-1), On(0)], [On(0), On(-1)], [On(0), On(1)], [On(-1), On(-1)]):
        with pytest.raises(ra.RopeError):
            where(bad)


def test_python_functions_refuse_other_ranks_and_types():
    with pytest.raises(ra.RopeError):
        ra.rope_latent_attention_paged(zeros(0, 128), zeros(0, 16, 192), ints(0, 1), ints(0), 128, 0.1)
    with pytest.raises(ra.RopeError):
        ra.rope_latent_attention(zeros(0, 128), zeros(0, 2, 64), zeros(0, 64), zeros(0, 2, 64), 0.1)
    with pytest.raises(ra.RopeError):
        ra._pack(torch.zeros(1, 1, 1, 1, 1))
    with pytest.raises(ra.RopeError):
        ra._pack(torch.zeros(()))
    for dtype in (torch.float64, torch.int32, torch.bool, torch.float8_e4m3fn):
        assert ra._dtype_code(torch.zeros(2).to(dtype)) not in CODES.values()

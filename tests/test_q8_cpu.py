"""CPU tests of the boundary of the 8-bit paged cache's calls and of the calls on pages (no kernel runs
here): every refusal of the host checks, the calls that have nothing to do, views that must not be
refused, and what the Python functions refuse before the C call."""
import ctypes

import pytest
import torch

import rope_partial_inplace_amd as ra
from test_paged_latent_cpu import (BF16, F16, F32, HAS_GPU, INVALID, NULLPTR, OK, RUNTIME, Call, desc,
                                   ints, zeros)

I8, E4M3, I64 = torch.int8, torch.float8_e4m3fn, torch.int64
CODES = {F32: 0, F16: 1, BF16: 2, I64: 3, I8: 4, E4M3: 5}


def codes(*shape, dtype=I8):
    return torch.zeros(shape, dtype=torch.int8).view(dtype)


def described(t, **override):
    return desc(t, **{"dtype": CODES.get(t.dtype, 9), **override})


def packed(tensors):
    """Descriptions one after the other, as the calls on pages take their caches."""
    out = (ra.RopeTensor * max(1, len(tensors)))()
    for i, t in enumerate(tensors):
        out[i] = t if isinstance(t, ra.RopeTensor) else described(t)
    return ctypes.cast(out, ctypes.c_void_p)


class Q8Call(Call):
    def run(self, **change):
        a = {**self.args, **change}
        change = {n: described(a[n]) for n in self.names if isinstance(a[n], torch.Tensor)} | {
            n: a[n] for n in self.names if not isinstance(a[n], torch.Tensor)}
        return super().run(**change)

    def changed(self, name, **override):
        return self.run(**{name: described(self.args[name], **override)})


class AppendQ8(Q8Call):
    fn = "rope_append_paged_cache_q8"
    names = ("positions", "query", "key", "value", "table", "page_table", "seq_lens", "offsets",
             "q_start", "k_start", "neox", "query_out", "key_cache", "value_cache", "key_scales",
             "value_scales", "stream")

    def tensors(self):
        return dict(positions=ints(6), query=zeros(6, 4, 96), key=zeros(6, 2, 128),
                    value=zeros(6, 2, 64), table=zeros(50, 64), page_table=ints(3, 4),
                    seq_lens=ints(3), offsets=ints(4), query_out=zeros(6, 4, 96),
                    key_cache=codes(5, 16, 2, 128), value_cache=codes(5, 16, 2, 64),
                    key_scales=zeros(5, 4, 2, dtype=F32), value_scales=zeros(5, 4, 2, dtype=F32))

    def plain(self):
        return dict(q_start=32, k_start=64, neox=1, stream=None)


class Attention(Q8Call):
    fn = "rope_attention_paged_q8"
    names = ("query", "key_cache", "value_cache", "key_scales", "value_scales", "page_table",
             "seq_lens", "offsets", "scale", "out", "lse", "workspace", "workspace_bytes", "stream")

    def tensors(self):
        need = ra.LIB.rope_attention_paged_q8_workspace(6, 4, 2, 128, 3)
        self.memory = torch.zeros(need + 64, dtype=torch.uint8)
        return dict(query=zeros(6, 4, 128), key_cache=codes(5, 16, 2, 128),
                    value_cache=codes(5, 16, 2, 128), key_scales=zeros(5, 4, 2, dtype=F32),
                    value_scales=zeros(5, 4, 2, dtype=F32), page_table=ints(3, 4), seq_lens=ints(3),
                    offsets=ints(4), out=zeros(6, 4, 128), lse=zeros(6, 4, dtype=F32))

    def plain(self):
        return dict(scale=0.1, workspace=self.memory.data_ptr(), workspace_bytes=self.memory.numel(),
                    stream=None)


class PageCall(Q8Call):
    """caches: a list of tensors or descriptions."""

    def caches(self):
        return [zeros(20, 16, 2, 64), codes(20, 16, 2, 64), zeros(20, 4, 2, dtype=F32)]

    def __init__(self):
        super().__init__()
        self.args["caches"] = self.caches()

    def run(self, **change):
        caches = change.get("caches", self.args["caches"])
        if isinstance(caches, list):
            self.held = caches
            change = {"num_caches": len(caches), **change, "caches": packed(caches)}
        return super().run(**change)


class Copy(PageCall):
    fn = "rope_copy_pages"
    names = ("sources", "targets", "caches", "num_caches", "stream")

    def tensors(self):
        return dict(sources=ints(7), targets=ints(7))

    def plain(self):
        return dict(num_caches=3, stream=None)


class Fork(PageCall):
    fn = "rope_fork_pages"
    names = ("page_table", "seq_lens", "parents", "grow", "ref_counts", "page_size", "caches",
             "num_caches", "page_table_out", "seq_lens_out", "ref_counts_out", "shortage", "workspace",
             "workspace_bytes", "stream")

    def tensors(self):
        need = ra.LIB.rope_fork_pages_workspace(3, 5, 20)
        self.memory = torch.zeros(need + 64, dtype=torch.uint8)
        return dict(page_table=ints(3, 4), seq_lens=ints(3), parents=ints(5), grow=ints(5),
                    ref_counts=ints(20), page_table_out=ints(5, 4), seq_lens_out=ints(5),
                    ref_counts_out=ints(20), shortage=ints(1))

    def plain(self):
        at = (self.memory.data_ptr() + 15) // 16 * 16
        return dict(page_size=16, num_caches=3, workspace=at, workspace_bytes=self.memory.numel() - 16,
                    stream=None)


class Compact(PageCall):
    fn = "rope_compact_pages"
    names = ("page_table", "ref_counts", "caches", "num_caches", "page_table_out", "ref_counts_out",
             "page_map", "live", "workspace", "workspace_bytes", "stream")

    def tensors(self):
        need = ra.LIB.rope_compact_pages_workspace(20)
        self.memory = torch.zeros(need + 64, dtype=torch.uint8)
        return dict(page_table=ints(3, 4), ref_counts=ints(20), page_table_out=ints(3, 4),
                    ref_counts_out=ints(20), page_map=ints(20), live=ints(1))

    def plain(self):
        at = (self.memory.data_ptr() + 15) // 16 * 16
        return dict(num_caches=3, workspace=at, workspace_bytes=self.memory.numel() - 16, stream=None)


CALLS = {"append": AppendQ8, "attention": Attention, "copy": Copy, "fork": Fork, "compact": Compact}
OPTIONAL = {"append": {"offsets"}, "attention": {"offsets", "lse"}, "copy": set(), "fork": {"grow"},
            "compact": set()}
OUTPUTS = {"append": ("query_out", "key_cache", "value_cache", "key_scales", "value_scales"),
           "attention": ("out", "lse"), "copy": (),
           "fork": ("page_table_out", "seq_lens_out", "ref_counts_out", "shortage"),
           "compact": ("page_table_out", "ref_counts_out", "page_map", "live")}
TENSORS = [(c, n) for c in CALLS for n in CALLS[c]().tensors()]
# dimensions of a tensor that may be longer without another's being
FREE = {("append", "table"): (0,), ("append", "page_table"): (1,), ("attention", "page_table"): (1,),
        ("fork", "page_table_out"): (1,)}


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
    mine = CODES[t.dtype]
    for dtype in {-1, 0, 3, 4, 5, 6, 9} - {mine}:
        assert c.changed(name, dtype=dtype) == INVALID, dtype
    for d in range(t.dim()):
        shape = list(t.shape)
        if d not in FREE.get((call, name), ()):
            shape[d] += 1
            assert c.changed(name, shape=shape) == INVALID, (d, shape)
        shape[d] = -1
        assert c.changed(name, shape=shape) == INVALID
        if t.shape[d] > 1:
            stride = list(t.stride())
            stride[d] = -stride[d]
            assert c.changed(name, stride=stride) == INVALID
            stride[d] = 1 << 62
            assert c.changed(name, stride=stride) == INVALID
    if t.dtype not in (I64, F32) and t.dim() > 1:
        stride = [2 * s for s in t.stride()]
        assert c.changed(name, stride=stride) == INVALID  # no unit inner stride


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in OUTPUTS[c]])
def test_outputs_overlap_nothing(call, name):
    c = CALLS[call]()
    own = {("append", "query_out"): "query", ("fork", "ref_counts_out"): "ref_counts",
           ("compact", "ref_counts_out"): "ref_counts",
           ("compact", "page_table_out"): "page_table"}.get((call, name))
    for other, t in c.args.items():
        if not isinstance(t, torch.Tensor) or other in (name, own):
            continue
        first = t.data_ptr()
        last = first + (t.numel() - 1) * t.element_size() // 16 * 16
        assert c.changed(name, data=first) == INVALID, other
        assert c.changed(name, data=last // 16 * 16) == INVALID, other
    for cache in c.args.get("caches", []):
        assert c.changed(name, data=cache.data_ptr()) == INVALID
    if "workspace" in c.args:
        assert c.changed(name, data=c.args["workspace"]) == INVALID
    out = c.args[name]
    if out.dim() > 1 or out.numel() > 1:
        stride = list(out.stride())
        stride[0] = 0
        assert c.changed(name, stride=stride) == INVALID  # reaches elements twice (or not contiguous)
    if own and out.dim() > 1:  # its own input: the same view only
        t = c.args[own]
        stride = list(t.stride())
        stride[0] *= 2
        assert c.run(**{name: described(t, stride=stride)}) == INVALID


@pytest.mark.parametrize("call", ["attention", "fork", "compact"])
def test_workspaces(call):
    c = CALLS[call]()
    need = {"attention": lambda: ra.LIB.rope_attention_paged_q8_workspace(6, 4, 2, 128, 3),
            "fork": lambda: ra.LIB.rope_fork_pages_workspace(3, 5, 20),
            "compact": lambda: ra.LIB.rope_compact_pages_workspace(20)}[call]()
    assert c.run(workspace=None) == NULLPTR
    for size in (need - 1, 0, -1):
        assert c.run(workspace_bytes=size) == INVALID
    assert c.run(workspace=c.args["workspace"] + 8) == INVALID
    tensors = [t for t in c.args.values() if isinstance(t, torch.Tensor)] + c.args.get("caches", [])
    for t in tensors:
        for at in (t.data_ptr(), t.data_ptr() - need):
            at = at // 16 * 16 + (16 if at < t.data_ptr() else 0)
            assert c.run(workspace=at, workspace_bytes=need) == INVALID


def test_workspace_sizes():
    big = 2 ** 62
    attention = ra.LIB.rope_attention_paged_q8_workspace
    for args in ((0, 4, 2, 128, 1), (1, 0, 2, 128, 1), (1, 4, 0, 128, 1), (1, 4, 2, 0, 1),
                 (1, 4, 2, 128, 0), (-1, 4, 2, 128, 1), (1, 4, 3, 128, 1), (big, 4, 2, 128, 1),
                 (1, big, 2, 128, 1), (1, 4, 2, big, 1)):
        assert attention(*args) == 0
    assert 0 < attention(1, 16, 1, 128, 1) < attention(1, 17, 1, 128, 1) < attention(1, 33, 1, 128, 1)
    assert attention(4, 4, 4, 64, big) == attention(4, 4, 4, 64, 4)
    fork, compact = ra.LIB.rope_fork_pages_workspace, ra.LIB.rope_compact_pages_workspace
    assert fork(0, 0, 0) > 0 and compact(0) > 0
    assert fork(3, 5, 100000) >= 100000 * 4 + 5 * 32 + 3 * 12 and compact(10 ** 6) >= 8 * 10 ** 6
    for args in ((-1, 1, 1), (1, -1, 1), (1, 1, -1), (big, 1, 1), (1, big, 1), (1, 1, big)):
        assert fork(*args) == 0
    assert compact(-1) == compact(big) == 0


def test_append_options():
    c = AppendQ8()
    assert c.run(query=None) == NULLPTR and c.run(query_out=None) == NULLPTR
    for start in (-1, 33, 1 << 62):
        assert c.run(q_start=start) == INVALID
    for start in (-1, 65, -(1 << 62)):
        assert c.run(k_start=start) == INVALID
    for table in (zeros(0, 64), zeros(50, 0), zeros(50, 63), zeros(50, 98)):
        assert c.run(table=table) == INVALID
    for blocks in (0, 3, 5, 32):  # of 16 rows
        assert c.run(key_scales=zeros(5, blocks, 2, dtype=F32),
                     value_scales=zeros(5, blocks, 2, dtype=F32)) == INVALID
    assert c.run(value_cache=codes(5, 16, 2, 64, dtype=E4M3)) == INVALID  # codes of two types
    assert c.run(offsets=None, seq_lens=ints(4), page_table=ints(4, 4)) == INVALID  # 6 % 4
    assert c.run(offsets=None, seq_lens=ints(0), page_table=ints(0, 4)) == INVALID
    huge = 1 << 30
    assert c.changed("page_table", shape=(3, huge), stride=(0, 0)) == INVALID
    assert c.changed("page_table", shape=(3, huge // 16), stride=(0, 0)) == INVALID
    q = c.args["query"]
    assert c.run(query_out=described(q, data=q.data_ptr() + 16)) == INVALID


def test_attention_options():
    c = Attention()
    for scale in (float("nan"), float("inf"), -float("inf"), 1e39):
        assert c.run(scale=scale) == INVALID
    for width in (32, 96, 192, 512):
        assert c.run(query=zeros(6, 4, width), out=zeros(6, 4, width), key_cache=codes(5, 16, 2, width),
                     value_cache=codes(5, 16, 2, width)) == INVALID
    assert c.run(query=zeros(6, 5, 128), out=zeros(6, 5, 128), lse=zeros(6, 5, dtype=F32)) == INVALID
    assert c.run(value_cache=codes(5, 16, 2, 128, dtype=E4M3)) == INVALID
    assert c.run(query=zeros(6, 4, 128, dtype=F32), out=zeros(6, 4, 128, dtype=F32)) == INVALID
    assert c.run(offsets=None, seq_lens=ints(4), page_table=ints(4, 4)) == INVALID
    for name in ("query", "key_cache", "value_cache", "out"):
        assert c.changed(name, data=c.args[name].data_ptr() + 2) == INVALID
    for name in ("key_cache", "value_cache"):
        stride = list(c.args[name].stride())
        stride[1] += 8
        assert c.changed(name, stride=stride) == INVALID
        stride[1] = 1 << 24  # tokens too far apart
        assert c.changed(name, stride=stride) == INVALID


def test_page_options():
    for call in (Copy, Fork, Compact):
        c = call()
        assert c.run(caches=None, num_caches=2) == NULLPTR
        for n in (-1, (1 << 16) + 1):
            assert c.run(caches=packed(c.caches()), num_caches=n) == INVALID
        x = zeros(20, 16, 2, 64)
        for bad in (described(x, shape=(19, 16, 2, 64)),       # other pages than the others
                    described(x, dtype=9), described(x, ndim=0), described(x, ndim=5),
                    described(x, stride=(2048, 64, 1024, 1), shape=(20, 8, 2, 64)),  # gaps in a page
                    described(x, stride=(1024, 128, 64, 1)),   # pages overlap
                    described(x, stride=(0, 128, 64, 1)),
                    described(x, stride=(2048, 128, 64, 2)),
                    described(x, stride=(-2048, 128, 64, 1))):
            assert c.run(caches=[zeros(20, 16, 2, 64), bad]) == INVALID
        assert c.run(caches=[described(x, data=None)]) == NULLPTR
        assert c.run(caches=[x, x]) == INVALID
        assert c.run(caches=[x, described(x, data=x.data_ptr() + 20 * 4096 - 64)]) == INVALID
        assert c.run(caches=[described(x, shape=(20, 1 << 31, 2, 64), stride=(1 << 38, 128, 64, 1),
                                       dtype=4, data=x.data_ptr() + 1)]) == INVALID  # words of a byte
    c = Fork()
    for size in (0, -1, 1 << 30):
        assert c.run(page_size=size) == INVALID
    assert c.run(page_table_out=ints(5, 3)) == INVALID  # narrower than what it continues
    assert c.run(page_size=1 << 28) == INVALID          # tokens of a row past 2^30
    c = Copy()
    assert c.run(targets=ints(6)) == INVALID
    assert c.run(caches=[c.args["sources"].view(7, 1)]) == INVALID


def test_calls_without_work_launch_nothing():
    c = AppendQ8()
    assert c.run(positions=ints(0), query=zeros(0, 4, 96), key=zeros(0, 2, 128), value=zeros(0, 2, 64),
                 query_out=zeros(0, 4, 96), offsets=ints(4)) == OK
    none = dict(query=None, query_out=None)
    assert c.run(key_cache=codes(0, 16, 2, 128), value_cache=codes(0, 16, 2, 64),
                 key_scales=zeros(0, 4, 2, dtype=F32), value_scales=zeros(0, 4, 2, dtype=F32),
                 **none) == OK  # a cache without pages takes nothing
    assert c.run(offsets=ints(1), seq_lens=ints(0), page_table=ints(0, 4), **none) == OK
    assert c.run(page_table=ints(3, 0), **none) == OK
    assert c.run(key=zeros(6, 0, 128), value=zeros(6, 0, 64), key_cache=codes(5, 16, 0, 128),
                 value_cache=codes(5, 16, 0, 64), key_scales=zeros(5, 4, 0, dtype=F32),
                 value_scales=zeros(5, 4, 0, dtype=F32), **none) == OK
    c = Attention()
    assert c.run(query=zeros(0, 4, 128), out=zeros(0, 4, 128), lse=zeros(0, 4, dtype=F32)) == OK
    assert c.run(query=zeros(6, 0, 128), out=zeros(6, 0, 128), lse=zeros(6, 0, dtype=F32),
                 workspace=None, workspace_bytes=0) == OK
    assert c.run(offsets=ints(1), seq_lens=ints(0), page_table=ints(0, 4), workspace=None,
                 workspace_bytes=0) == OK
    c = Copy()
    assert c.run(sources=ints(0), targets=ints(0)) == OK
    assert c.run(caches=[]) == OK and c.run(caches=[zeros(20, 0, 4), zeros(20, 16, 0)]) == OK


@pytest.mark.skipif(HAS_GPU, reason="reaches the launch, with host buffers")
def test_views_that_are_accepted():
    c = AppendQ8()
    qkv = zeros(6, 8, 160)  # columns of one projection
    assert c.run(query=qkv[:, :4, :96], key=qkv[:, 4:6, :128], value=qkv[:, 6:, :64]) == RUNTIME
    both = codes(5, 16, 2, 192)  # keys and values of a row side by side
    assert c.run(key_cache=both[..., :128], value_cache=both[..., 128:]) == RUNTIME
    both = codes(5, 2, 2, 16, 128)  # keys and values of a page in turn, heads before rows
    assert c.run(key_cache=both[:, 0].transpose(1, 2),
                 value_cache=both[:, 1, ..., :64].transpose(1, 2)) == RUNTIME
    s = zeros(5, 2, 2, 4, dtype=F32)
    assert c.run(key_scales=s[:, 0].transpose(1, 2), value_scales=s[:, 1].transpose(1, 2)) == RUNTIME
    assert c.run(query_out=c.args["query"]) == RUNTIME  # in place
    assert c.run(query=None, query_out=None) == RUNTIME
    assert c.run(offsets=None) == RUNTIME
    e = dict(key_cache=codes(5, 16, 2, 128, dtype=E4M3), value_cache=codes(5, 16, 2, 64, dtype=E4M3))
    assert c.run(**e) == RUNTIME
    c = Attention()
    assert c.run(lse=None, offsets=None) == RUNTIME
    assert c.run(scale=0.0) == RUNTIME and c.run(scale=-1.0) == RUNTIME
    wide = zeros(6, 4, 256)
    assert c.run(query=wide[..., :128]) == RUNTIME
    for call in (Copy, Fork, Compact):
        c = call()
        both = zeros(20, 2, 16, 2, 64)
        assert c.run(caches=[both[:, 0], both[:, 1]]) == RUNTIME
        assert c.run(caches=[zeros(20, 2, 16, 64).transpose(1, 2), zeros(20)]) == RUNTIME
        assert c.run(caches=[ints(20, 3), codes(20, 5, dtype=E4M3)]) == RUNTIME
        assert c.run(caches=[zeros(20, 4) for _ in range(200)]) == RUNTIME
    c = Fork()
    assert c.run(caches=[], grow=None) == RUNTIME
    assert c.run(ref_counts_out=c.args["ref_counts"]) == RUNTIME
    assert c.run(page_table_out=ints(5, 9)) == RUNTIME
    c = Compact()
    assert c.run(caches=[], ref_counts_out=c.args["ref_counts"],
                 page_table_out=c.args["page_table"]) == RUNTIME


def python_calls():
    a, t = AppendQ8().args, Attention().args
    c, f, m = Copy(), Fork(), Compact()
    yield lambda: ra.rope_append_paged_cache_q8(a["positions"], a["key"], a["value"], a["key_cache"],
                                                a["value_cache"], a["key_scales"],
                                                a["value_scales"], a["page_table"], a["seq_lens"],
                                                a["table"])
    yield lambda: ra.rope_attention_paged_q8(t["query"], t["key_cache"], t["value_cache"],
                                             t["key_scales"], t["value_scales"], t["page_table"],
                                             t["seq_lens"], 0.1)
    yield lambda: ra.rope_copy_pages(c.args["sources"], c.args["targets"], c.caches())
    yield lambda: ra.rope_fork_pages(f.args["page_table"], f.args["seq_lens"], f.args["parents"],
                                     f.args["ref_counts"], 16)
    yield lambda: ra.rope_compact_pages(m.args["page_table"], m.args["ref_counts"])
    yield lambda: ra.PageCaches(c.caches())


@pytest.mark.parametrize("n", range(6))
def test_python_functions_refuse_host_tensors(n):
    with pytest.raises(ra.RopeError) as e:
        list(python_calls())[n]()
    assert e.value.code == INVALID and "GPU memory" in str(e.value)


def test_python_functions_refuse_other_ranks():
    a, t, f = AppendQ8().args, Attention().args, Fork().args
    with pytest.raises(ra.RopeError):
        ra.rope_attention_paged_q8(zeros(0, 128), codes(0, 16, 2, 128), codes(0, 16, 2, 128),
                                   zeros(0, 4, 2, dtype=F32), zeros(0, 4, 2, dtype=F32), ints(0, 1),
                                   ints(0), 0.1)
    with pytest.raises(ra.RopeError):
        ra.rope_fork_pages(ints(0), ints(0), ints(0), ints(0), 16)
    with pytest.raises(ra.RopeError):
        ra.rope_compact_pages(ints(0, 1), ints(0, 1))
    assert a and t and f


def test_caches_on_two_devices_are_refused(monkeypatch):
    """Checked with a stand-in for the device of the list."""
    caches = ra.PageCaches([])
    caches.device = 1
    assert ra._page_caches(caches, 1) == (caches, 1) and ra._page_caches(caches, -1) == (caches, 1)
    with pytest.raises(ra.RopeError):
        ra._page_caches(caches, 0)

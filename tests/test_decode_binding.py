"""What the Python calls of the decode step hand to the library: traced on the CPU with stand-ins for tensors on a GPU,
the library and the stream."""
import pytest
import torch

BF = torch.bfloat16


class OnGpu:
    """A CPU tensor that says it lies on GPU `index`: what the binding reads of a tensor before it passes its address."""

    def __init__(self, t: torch.Tensor, index: int = 0):
        self.t, self.index = t, index

    def __getattr__(self, name):
        return getattr(self.t, name)

    is_cuda = True

    @property
    def device(self):
        return torch.device("cuda", self.index)

    def get_device(self):
        return self.index


def zeros(*shape, dtype=BF, index=0):
    return OnGpu(torch.zeros(*shape, dtype=dtype), index)


def expand(t: OnGpu, *shape):
    return OnGpu(t.t.expand(*shape), t.index)


class Library:
    """Records the calls and their arguments; every call succeeds.  (Handles of earlier tests may be collected meanwhile:
    their destruction goes to the library.)"""

    def __init__(self, real):
        self.calls, self.real = [], real

    def __getattr__(self, name):
        if name.endswith("_destroy"):
            return getattr(self.real(), name)
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def m(monkeypatch):
    import block_scaled_fp4_sqrt_gb300 as mod
    from block_scaled_fp4_sqrt_gb300 import decode
    library = Library(mod.lib)
    for at in (mod, decode):
        monkeypatch.setattr(at, "lib", lambda: library)
        monkeypatch.setattr(at, "_raw_stream", lambda stream: 0 if stream is None else int(stream))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    mod.library = library
    yield mod
    del mod.library


def cache(m, n_seqs=3, heads=2, head_dim=64):
    c = object.__new__(m.PagedKVCache)
    c.n_seqs, c.n_kv_heads, c.head_dim = n_seqs, heads, head_dim
    c.device, c._index, c._ref, c._workspace_bytes = torch.device("cuda", 0), 0, None, {}
    return c


# ---------------------------------------------------------------------------------------------- broadcast rows
def test_norm_passes_row_strides_and_refuses_broadcast_rows(m):
    """The library reads stride 0 as contiguous rows: a broadcast tensor would be read and written past its end."""
    w, wide, lone = zeros(64), zeros(4, 200), zeros(1, 64)
    x = OnGpu(wide.t[:, 72:136])
    m.moe_add_rms_norm(x, None, w, y=zeros(4, 64))
    args = m.library.calls[-1][1][0]
    assert (args.T, args.d, args.x_stride, args.y_stride) == (4, 64, 200, 64)
    m.moe_add_rms_norm(lone, expand(lone, 1, 64), w, y=lone)  # one row has no stride
    rows, calls = expand(lone, 4, 64), len(m.library.calls)
    full = zeros(4, 64)
    for kw in (dict(x=rows, residual=None, y=full), dict(x=full, residual=rows, y=full),
               dict(x=full, residual=None, y=rows), dict(x=full, residual=None, sum_out=rows)):
        with pytest.raises(ValueError, match="row"):
            m.moe_add_rms_norm(weight=w, **kw)
    u8 = torch.uint8
    with pytest.raises(ValueError):
        m.moe_add_rms_norm(full, None, w, y_q=expand(zeros(1, 64, dtype=u8), 4, 64), y_s=zeros(4, 2, dtype=u8))
    with pytest.raises(ValueError):
        m.moe_add_rms_norm(full, None, w, y_q=zeros(4, 64, dtype=u8), y_s=expand(zeros(1, 2, dtype=u8), 4, 2))
    assert len(m.library.calls) == calls


@pytest.mark.parametrize("L", [1, 2])
def test_append_and_attend_refuse_broadcast_rows(m, L):
    c = cache(m)
    full, fq = zeros(3, L, 2, 64), zeros(3, L, 4, 64)
    c.append(full, full)
    assert m.library.calls[-1][1][2] == 2 * 64
    calls = len(m.library.calls)
    for t in (expand(zeros(1, 1, 2, 64), 3, L, 2, 64), expand(zeros(1, L, 2, 64), 3, L, 2, 64)):
        for args in ((t, full), (full, t)):
            with pytest.raises(ValueError):
                c.append(*args)
    for q in (expand(zeros(1, 1, 4, 64), 3, L, 4, 64), expand(zeros(1, L, 4, 64), 3, L, 4, 64)):
        for args in ((q, fq), (fq, q)):
            with pytest.raises(ValueError):
                c.attend(*args)
    one = cache(m, n_seqs=1)
    if L > 1:
        with pytest.raises(ValueError):
            one.append(expand(zeros(1, 1, 2, 64), 1, L, 2, 64), zeros(1, L, 2, 64))
    assert len(m.library.calls) == calls


# ---------------------------------------------------------------------------------------------- the few-token layer
def layer(m, d=256, k=2, hash_table=None):
    lay = object.__new__(m.MoELayer)
    lay.d, lay.k, lay.device, lay.hash_table, lay._handles = d, k, torch.device("cuda", 0), hash_table, []
    lay.h = lay.h_shared = None
    lay.router_w = lay.router_bias = None
    lay.resident_router = True
    return lay


def test_forward_few_passes_what_fits_and_refuses_the_rest(m):
    """The kernel writes dense rows of the batch's size into out, topk_ids and topk_w, whatever they are."""
    lay, x, i32, f32 = layer(m), zeros(3, 256), torch.int32, torch.float32
    good = dict(out=zeros(3, 256), topk_ids=zeros(3, 2, dtype=i32), topk_w=zeros(3, 2, dtype=f32))
    assert lay.forward_few(x, **good) is good["out"]
    assert [c[0] for c in m.library.calls] == ["moe_forward_few"]
    lay.forward_few(x, token_ids=zeros(5, dtype=i32), **good)  # the first T of a longer list
    lay.forward_few(zeros(0, 256), out=zeros(0, 256))
    six = zeros(6, 256)  # dense memory of the right size, kept in another shape: two requests of three rows
    lay.forward_few(six, zeros(2, 3, dtype=i32), zeros(2, 3, 256), zeros(2, 3, 2, dtype=i32), zeros(2, 3, 2, dtype=f32))
    calls = len(m.library.calls)
    for kw in (dict(x=zeros(3, 128)), dict(x=zeros(3, 256, dtype=f32)), dict(x=OnGpu(torch.zeros(3, 512, dtype=BF)[:, ::2])),
               dict(x=x.t), dict(out=zeros(2, 256)), dict(out=zeros(3, 256, dtype=f32)), dict(out=zeros(3, 264)),
               dict(out=expand(zeros(1, 256), 3, 256)), dict(topk_ids=zeros(3, 2, dtype=torch.int64)),
               dict(topk_ids=zeros(2, 2, dtype=i32)), dict(topk_ids=zeros(3, 1, dtype=i32)), dict(topk_ids=zeros(6, dtype=i32)),
               dict(topk_ids=OnGpu(torch.zeros(2, 3, dtype=i32).t())), dict(topk_w=zeros(3, 2, dtype=BF)),
               dict(topk_w=zeros(3, 2, dtype=f32).t), dict(topk_w=zeros(1, 2, dtype=f32)),
               dict(token_ids=zeros(3, dtype=torch.int64)), dict(token_ids=zeros(2, dtype=i32)),
               dict(token_ids=OnGpu(torch.zeros(6, dtype=i32)[::2]))):
        with pytest.raises(ValueError):
            lay.forward_few(**{"x": x, **good, **kw})
    assert len(m.library.calls) == calls


# ---------------------------------------------------------------------------------------------- streams
def test_results_are_allocated_on_the_stream_that_writes_them(m, monkeypatch):
    """Memory of the current stream's pool may still be in use there when a kernel on another stream writes it."""
    active, made = [], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            active.append(self.stream)

        def __exit__(self, *_):
            active.pop()

    def empty(*args, device=None, _real=torch.empty, **kw):
        made.append(active[-1] if active else None)
        return OnGpu(_real(*args, **kw))

    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch, "empty", empty)
    c, lay, x, q = cache(m), layer(m), zeros(3, 256), zeros(3, 1, 4, 64)
    monkeypatch.setattr(m.PagedKVCache, "_workspace", lambda *a: zeros(8, dtype=torch.uint8))
    for stream, want in ((None, None), (77, 77), (0, "default")):
        for call in (lambda: c.attend(q, stream=stream), lambda: lay.forward_few(x, stream=stream),
                     lambda: lay.forward(x, stream=stream)):
            made.clear()
            call()
            assert made == [want]
            raw = m.library.calls[-1][1][-1]
            assert (getattr(raw, "value", raw) or 0) == (stream or 0)


# ---------------------------------------------------------------------------------------------- attention workspaces
def test_attention_workspaces(m, monkeypatch):
    """One a stream for every cache and shape, a private one in a capture, the caller's where it is given; the counters are
    cleared, the rest is not."""
    from block_scaled_fp4_sqrt_gb300 import decode
    sizes, state, made = {(4, 1): 6000, (4, 2): 9000, (8, 1): 7000}, dict(stream=1, capturing=False), []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            self.before = state["stream"]
            state["stream"] = self.stream or self.before

        def __exit__(self, *_):
            state["stream"] = self.before

    def empty(shape, dtype=None, device=None, _real=torch.empty):
        t = torch.full(shape, 7, dtype=dtype) if dtype is torch.uint8 else _real(shape, dtype=dtype)
        made.append((state["stream"], t))
        return Memory(t)

    class Memory(OnGpu):
        def __getitem__(self, at):
            return self.t[at]

    def size(ref, heads, L):
        return sizes[heads, L]

    m.library.moe_paged_attention_workspace = size
    m.library.moe_paged_attention = lambda ref, a, stream: used.append((a._obj.workspace, a._obj.workspace_bytes, stream)) or 0
    used = []
    monkeypatch.setattr(decode, "_WORKSPACES", {})
    monkeypatch.setattr(decode, "_raw_stream", lambda stream: state["stream"] if stream is None else stream)
    monkeypatch.setattr(m, "_raw_stream", lambda stream: state["stream"] if stream is None else stream)
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: state["capturing"], raising=False)
    monkeypatch.setattr(torch, "empty", empty)
    one, two = cache(m), cache(m)
    q1, q2, q8 = zeros(3, 1, 4, 64), zeros(3, 2, 4, 64), zeros(3, 1, 8, 64)

    def attend(c, q, **kw):
        made.clear()
        c.attend(q, out=q, **kw)
        return used[-1], list(made)

    (ws, n, stream), new = attend(one, q1)
    assert stream == 1 and n == 6000 and len(new) == 1 and new[0][0] == 1
    t, zero = new[0][1], m.MOE_ATTENTION_COUNTER_BYTES
    assert t.data_ptr() == ws and not t[:zero].any() and (t[zero:] == 7).all()
    assert attend(two, q1) == ((ws, 6000, 1), [])          # another cache: the same
    (ws2, n, _), new = attend(one, q2)                     # a larger call: a larger one
    assert n == 9000 and len(new) == 1
    assert attend(two, q8) == ((ws2, 9000, 1), []) and attend(one, q1) == ((ws2, 9000, 1), [])
    (ws3, n, stream), new = attend(one, q1, stream=5)      # another stream: its own, made there
    assert stream == 5 and n == 6000 and ws3 != ws2 and [s for s, _ in new] == [5]
    state["capturing"] = True
    (ws4, n, _), new = attend(one, q1)                     # in a capture: one that no other call uses
    assert n == 6000 and ws4 not in (ws2, ws3) and len(new) == 1
    assert len(attend(one, q1, stream=5)[1]) == 1
    mine = zeros(9000, dtype=torch.uint8)
    assert attend(one, q2, workspace=mine) == ((mine.data_ptr(), 9000, 1), [])
    state["capturing"] = False
    assert attend(one, q1) == ((ws2, 9000, 1), [])
    for bad in (zeros(9000, dtype=BF), OnGpu(torch.zeros(9000, dtype=torch.uint8)[::2]), zeros(9000, dtype=torch.uint8, index=1)):
        with pytest.raises(ValueError):
            one.attend(q1, out=q1, workspace=bad)


# ---------------------------------------------------------------------------------------------- devices
def test_calls_refuse_tensors_of_another_device(m, monkeypatch):
    """A call runs on the current device: neither another device's tensors nor a mixture reach the library."""
    def there(*shape, dtype=BF):
        return zeros(*shape, dtype=dtype, index=1)

    x, w, q, lay, c = zeros(4, 64), zeros(64), zeros(3, 1, 4, 64), layer(m), cache(m)
    u8, f32, i32 = torch.uint8, torch.float32, torch.int32
    mixed = [lambda: m.moe_add_rms_norm(x, None, there(64), y=x), lambda: m.moe_add_rms_norm(x, there(4, 64), w, y=x),
             lambda: m.moe_add_rms_norm(x, None, w, y=there(4, 64)), lambda: m.moe_add_rms_norm(x, None, w, sum_out=there(4, 64)),
             lambda: m.moe_add_rms_norm(x, None, w, y_q=there(4, 64, dtype=u8), y_s=zeros(4, 2, dtype=u8)),
             lambda: m.moe_add_rms_norm(x, None, w, y_q=zeros(4, 64, dtype=u8), y_s=there(4, 2, dtype=u8)),
             lambda: c.append(there(3, 1, 2, 64), zeros(3, 1, 2, 64)), lambda: c.attend(there(3, 1, 4, 64)),
             lambda: c.attend(q, out=there(3, 1, 4, 64)), lambda: c.attend(q, out=q, lse=there(3, 1, 4, dtype=f32)),
             lambda: lay.forward_few(zeros(3, 256), out=there(3, 256)),
             lambda: lay.forward_few(zeros(3, 256), out=zeros(3, 256), topk_ids=there(3, 2, dtype=i32)),
             lambda: lay.forward_few(zeros(3, 256), out=zeros(3, 256), topk_w=there(3, 2, dtype=f32)),
             lambda: lay.forward_few(zeros(3, 256), out=zeros(3, 256), token_ids=there(3, dtype=i32))]
    all_there = [lambda: m.moe_add_rms_norm(there(4, 64), None, there(64), y=there(4, 64)),
                 lambda: lay.forward_few(there(3, 256), out=there(3, 256))]
    new = zeros(3, 1, 2, 64)
    here = [lambda: m.moe_add_rms_norm(x, None, w, y=x), lambda: c.append(new, new),
            lambda: lay.forward_few(zeros(3, 256), out=zeros(3, 256))]
    for call in mixed + all_there:
        with pytest.raises(ValueError):
            call()
    assert not m.library.calls
    for call in here:
        call()
    assert len(m.library.calls) == 3
    m.library.calls.clear()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)  # the tensors' device is not the current one
    for call in here + [lambda: c.attend(q, out=q)]:
        with pytest.raises(ValueError, match="current device"):
            call()
    assert not m.library.calls

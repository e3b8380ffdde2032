"""Which buffers the layer objects keep (no GPU needed: the library's calls
are replaced by ones that allocate alike on the CPU)."""
import pytest
import torch

import routing_grouped_gemm_router_amd as moe

E, K, D, H = 8, 2, 64, 32
MIB = 1 << 20


@pytest.fixture
def capture(monkeypatch):
    """A switch: whether the current stream is being captured."""
    on = [False]
    monkeypatch.setattr(moe, "_capturing", lambda index: on[0])
    return on


def test_a_captured_size_stays(capture):
    s = moe._Sizes()
    fill = lambda key, n: s.at(key).setdefault("t", torch.empty(n, dtype=torch.uint8)).data_ptr()
    big = 2 * moe._KEPT_BYTES
    at = {}
    for key in (1, 2):
        at[key] = fill(key, big)
        capture[0] = True
        moe._mark(s.at(key), 0)
        capture[0] = False
    for key in range(3, 9):
        fill(key, big)
        moe._mark(s.at(key), 0)
        assert set(s._all) == {1, 2, key}                  # and of the others the last alone
    assert fill(1, big) == at[1] and fill(2, big) == at[2]


def test_small_sizes_stay_up_to_a_limit(capture):
    s = moe._Sizes()
    fill = lambda key, n: s.at(key).setdefault("d", dict(t=torch.empty(n, dtype=torch.uint8)))["t"].data_ptr()
    at = {key: fill(key, 16 * MIB) for key in range(4)}
    assert all(fill(key, 16 * MIB) == at[key] for key in range(4))
    fill(4, 16 * MIB)                                      # four of 16 MiB beside the last
    assert sorted(s._all) == [0, 1, 2, 3, 4]
    fill(5, 16 * MIB)                                      # the one that was used longest ago goes
    assert sorted(s._all) == [1, 2, 3, 4, 5]
    fill(6, 100 * MIB)
    assert sorted(s._all) == [2, 3, 4, 5, 6]
    fill(7, 1)                                             # the large one goes, small ones stay
    assert sorted(s._all) == [2, 3, 4, 5, 7]
    s.at(8)                                                # a refused call leaves nothing
    s.at(7)
    assert sorted(s._all) == [3, 4, 5, 7]                  # a byte and 64 MiB are too many


class _Device:
    def __init__(self, index):
        pass

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


@pytest.fixture
def on_cpu(monkeypatch, capture):
    """The layer objects' calls with tensors on the CPU and no arithmetic."""
    monkeypatch.setattr(moe, "_need_on", lambda t, shape, dtype, index, name: None)
    monkeypatch.setattr(torch.cuda, "device", _Device)
    monkeypatch.setattr(moe, "_check", lambda name, st: None)
    monkeypatch.setattr(moe, "_enqueue", lambda name, fn, index, *args: None)
    monkeypatch.setattr(moe, "_stream", lambda: 0)
    monkeypatch.setattr(moe, "_act_matrix",
                        lambda x, name: (x.shape[0], x.shape[1], moe.MOE_BF16, -1))
    monkeypatch.setattr(moe, "_need_ws", lambda ws, nbytes, like, gpu: ws)
    monkeypatch.setattr(moe, "_need", lambda t, shape, dtype, name: None)

    class Lib:
        def __getattr__(self, name):
            return getattr(lib, name) if name.endswith("_size") else lambda *args: 0

    lib = moe._lib
    monkeypatch.setattr(moe, "_lib", Lib())
    return capture


def _w4():
    return moe.MoELayerW4(torch.zeros(E, 2 * H, D), torch.zeros(E, D, H), K)


def _w4_step(layer, T):
    layer.forward(torch.zeros(T, D, dtype=torch.bfloat16), torch.zeros(T, E))
    return [t.data_ptr() for t in (layer.out, *layer.route.values())]


def test_w4_layer_keeps_its_buffers(on_cpu):
    """The addresses at a T are the same after calls at others."""
    layer = _w4()
    first = {T: _w4_step(layer, T) for T in (1, 4, 64)}
    assert first == {T: _w4_step(layer, T) for T in (1, 4, 64)}
    # sizes above what is kept: captured ones stay, in whatever order they come
    big = {}
    for T in (300000, 300001):
        _w4_step(layer, T)
        on_cpu[0] = True
        big[T] = _w4_step(layer, T)
        on_cpu[0] = False
    for T in (300002, 300003, 1):
        _w4_step(layer, T)
    assert big == {T: _w4_step(layer, T) for T in big}
    assert (300002, layer.w1q.get_device()) not in layer._sizes._all


def test_norm_keeps_its_buffers(on_cpu):
    norm = moe.LayerNorm(torch.zeros(D), torch.zeros(D), act8=True)

    def step(T, res):
        x = torch.zeros(T, D)
        norm.forward(x, x if res else None)
        norm.backward(x)
        return [t.data_ptr() for t in moe._tensors(dict(norm._out, g=norm.grads))]

    sizes = [(1, False), (1, True), (7, True)]
    first = {s: step(*s) for s in sizes}
    assert first == {s: step(*s) for s in sizes}


def test_norm_captured_in_its_backward_alone(on_cpu):
    """An eager forward and a captured backward: what the forward left is read at every replay."""
    norm = moe.LayerNorm(torch.zeros(D), None)
    x = torch.zeros(400000, D)
    norm.forward(x)
    on_cpu[0] = True
    norm.backward(x)
    on_cpu[0] = False
    at = (norm._out["mean"].data_ptr(), norm.grads["dx"].data_ptr())
    for T in (400001, 400002):
        norm.forward(torch.zeros(T, D))
        norm.backward(torch.zeros(T, D))
    norm.forward(x)
    norm.backward(x)
    assert at == (norm._out["mean"].data_ptr(), norm.grads["dx"].data_ptr())


def test_norm_adds_to_gradients_of_one_size_only(on_cpu):
    """Gradients of another size in between are not added to: refused as ever,
    though the buffers of the first size are still there."""
    norm = moe.LayerNorm(torch.zeros(D), None)
    a, b = torch.zeros(3, D), torch.zeros(5, D)
    for x in (a, b):
        norm.forward(x)
        norm.backward(x)
    norm.forward(a)
    with pytest.raises(ValueError, match="earlier backward"):
        norm.backward(a, accumulate_dw=True)
    norm.backward(a)
    norm.backward(a, accumulate_dw=True)


def test_capture_is_asked_of_the_buffers_gpu(monkeypatch):
    """The stream that counts is the current one of the GPU that the buffers are on."""
    current, seen = [1], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    monkeypatch.setattr(moe, "_cur_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(moe, "_cur_capturing",
                        lambda: seen.append(current[0]) or current[0] == 0)
    assert moe._capturing(0) and not moe._capturing(1) and seen == [0, 1] and current == [1]


def test_w4_weights_stay_in_their_tensors(on_cpu):
    layer = _w4()
    at = lambda: [t.data_ptr() for t in (layer.w1q, layer.w1s, layer.w2q, layer.w2s)]
    first = at()
    layer.prepare_weights(torch.ones(E, 2 * H, D), torch.ones(E, D, H))
    assert at() == first


@pytest.mark.parametrize("s1,s2", [((E, 2 * H, 2 * D), (E, 2 * D, H)), ((E, 2 * H, D), (E, D, 2 * H)),
                                   ((E + 1, 2 * H, D), (E + 1, D, H))])
def test_w4_weights_of_other_sizes_are_refused(on_cpu, monkeypatch, s1, s2):
    """Before either of the two is written."""
    layer, written = _w4(), []

    def need_on(t, shape, dtype, index, name):
        if tuple(t.shape) != shape:
            raise ValueError(name)

    monkeypatch.setattr(moe, "_need_on", need_on)
    monkeypatch.setattr(moe, "moe_w4_quantize", lambda *args: written.append(args))
    with pytest.raises(ValueError):
        layer.prepare_weights(torch.ones(s1), torch.ones(s2))
    assert not written


def _layer(kind):
    w = torch.zeros(E, 2 * H, D), torch.zeros(E, D, H)
    if kind == "padded":
        return moe.MoELayerPadded(*w, K, 8)
    opts = dict(aux_alpha=0.1, scratch={}, **({kind.split()[1]: True} if " " in kind else {}))
    return (moe.MoELayerMX if kind.startswith("mxfp8") else moe.MoELayer)(*w, K, **opts)


def _layer_step(layer, T, kind):
    x = torch.zeros(T, D, dtype=torch.bfloat16 if kind.startswith("mxfp8") else torch.float32)
    layer.forward(x, torch.zeros(T, E))
    layer.backward(x)
    own = {n: v for n, v in layer._buf["tensors"].items()}
    assert all(getattr(layer, n) is v for n, v in own.items())
    return [t.data_ptr() for t in moe._tensors(dict(layer._buf, grads=layer.grads))]


KINDS = ["plain", "plain act8", "plain recompute", "mxfp8", "mxfp8 act8", "mxfp8 recompute", "padded"]


@pytest.fixture
def layers_on_cpu(on_cpu, monkeypatch):
    """on_cpu for the layers with a backward."""
    monkeypatch.setattr(moe.MoELayer, "_check_input", lambda self, x, logits: None)
    for name in ("_act8_need", "_need_bytes", "moe_grouped_gemm", "moe_permute", "mxfp8_quantize"):
        monkeypatch.setattr(moe, name, lambda *args, **kw: None)
    monkeypatch.setattr(moe, "_p", lambda t: None)
    return on_cpu


@pytest.mark.parametrize("kind", KINDS)
def test_layers_keep_the_buffers_of_captured_sizes(layers_on_cpu, monkeypatch, kind):
    monkeypatch.setattr(moe, "_KEPT_BYTES", 0)
    layer, at = _layer(kind), {}
    for T in (96, 64):
        _layer_step(layer, T, kind)
        layers_on_cpu[0] = True
        at[T] = _layer_step(layer, T, kind)
        layers_on_cpu[0] = False
    for T in (128, 160):                                   # larger: the balancing loss's workspace too
        _layer_step(layer, T, kind)
        assert len(layer._sizes._all) == 3                 # of the others the last alone
    assert at == {T: _layer_step(layer, T, kind) for T in at}


@pytest.mark.parametrize("kind", KINDS)
def test_layers_add_to_gradients_of_one_size_only(layers_on_cpu, kind):
    layer = _layer(kind)
    x = {T: torch.zeros(T, D, dtype=torch.bfloat16 if kind.startswith("mxfp8") else torch.float32)
         for T in (64, 96)}
    forward = lambda T: layer.forward(x[T], torch.zeros(T, E))
    for T in (64, 96, 64):
        forward(T)
        with pytest.raises(ValueError, match="earlier backward"):
            layer.backward(x[T], accumulate_dw=True)
        layer.backward(x[T])
        forward(T)
        layer.backward(x[T], accumulate_dw=True)


def test_no_old_buffer_is_held_while_new_ones_are_made(layers_on_cpu, monkeypatch):
    """A call with another size has freed the last one's tensors before it allocates."""
    monkeypatch.setattr(moe, "_KEPT_BYTES", 0)
    import weakref
    layer = moe.MoELayer(torch.zeros(E, 2 * H, D), torch.zeros(E, D, H), K)
    _layer_step(layer, 64, "plain")
    old = [weakref.ref(t) for t in moe._tensors(layer._buf)]
    new, seen = layer._new, []
    monkeypatch.setattr(layer, "_new", lambda *a: seen.append([r() is None for r in old]) or new(*a))
    layer.forward(torch.zeros(96, D), torch.zeros(96, E))
    assert len(seen) == 1 and all(seen[0])


def test_mxfp8_weights_stay_in_their_tensors(layers_on_cpu):
    layer = _layer("mxfp8")
    at = lambda: [getattr(layer, n).data_ptr() for n in ("w1q", "w1s", "w1t", "w1ts", "w2q", "w2s",
                                                         "w2t", "w2ts")]
    first = at()
    layer.prepare_weights(torch.ones(E, 2 * H, D), torch.ones(E, D, H))
    assert at() == first
    layer.prepare_weights(torch.ones(E * 2 * H, D), torch.ones(E * D, H))
    assert at() == first
    for s1, s2 in (((E, 2 * H, 2 * D), (E, 2 * D, H)), ((E, 2 * H, D), (E, D, 2 * H))):
        with pytest.raises(RuntimeError):
            layer.prepare_weights(torch.ones(s1), torch.ones(s2))

"""CPU checks: the training calls launch on the current device, so tensors on
another one are refused before anything is launched.  Stand-in tensors report a
device, a stand-in library records its calls."""
import pytest
import torch


def _on(index):
    class Tensor(torch.Tensor):
        is_cuda = True
        device = torch.device("cuda", index)

        def get_device(self):
            return index
    return Tensor


ON = [_on(0), _on(1)]


def t(device, *shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(ON[device])


class Library:
    """Every call succeeds and is noted; sizes are the real library's."""

    def __init__(self, real):
        self._real, self.calls = real, []

    def __getattr__(self, name):
        if name in ("tb_grad_records", "tb_layer_norm_workspace", "tb_status_string"):
            return getattr(self._real, name)
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def tbl(monkeypatch):
    from patch_groupnorm_gb300 import build
    build.build()
    from patch_groupnorm_gb300 import tileblend
    monkeypatch.setattr(tileblend, "_lib", Library(tileblend._lib))
    monkeypatch.setattr(tileblend, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(tileblend, "_raw_stream", lambda device: 0)
    return tileblend


def _calls(tbl, d, **at):
    """Every training call with its tensors on device d, those named in
    ``at`` elsewhere."""
    def on(name, *shape, dtype=torch.float32):
        return t(at.get(name, d), *shape, dtype=dtype)
    x, w, s = on("x", 4, 8), on("w", 8), on("s", 4)
    patch, part = on("patch", 1, 4, 2, 2), on("part", 1, 1, 2, tbl.TB_GN_PARTS, 16, dtype=torch.uint8)
    grec, recs, norm = (on("grec", 1, 1, 4, tbl.TB_GN_PARTS, 2), on("recs", tbl.TB_GRAD_PARTS, dtype=torch.float64),
                        on("norm", 1))
    ws, grad = on("ws", 4 * 8 * 8, dtype=torch.uint8), on("grad", 8)
    c = on("c", 4)
    return {
        "layer_norm": lambda: tbl.tb_layer_norm(x, x, w, w, 1e-6, s, s),
        "layer_norm_backward": lambda: tbl.tb_layer_norm_backward(x, x, s, s, w, x, w, w, ws),
        "grad_stats": lambda: tbl.tb_grad_stats(tbl.GradTable([grad]), recs),
        "grad_norm": lambda: tbl.tb_grad_norm(recs, norm),
        "grad_clip": lambda: tbl.tb_grad_clip(tbl.GradTable([grad]), recs, 1.0, norm),
        "clip_grad_norm": lambda: tbl.clip_grad_norm([grad], 1.0, recs, norm),
        "gn_grad_stats": lambda: tbl.tb_patch_gn_grad_stats([patch], [patch], 2, part, 1, c, c, 1e-6, grec),
        "gn_grad_apply": lambda: tbl.tb_patch_gn_grad_apply([patch], [patch], [patch], 2, part, grec, 1, c, c, 1e-6),
        "gn_backward": lambda: tbl.patch_group_norm_backward([patch], [patch], 2, part, c, c, 1e-6, True, [patch], c, c,
                                                             grec),
    }


NAMES = ["layer_norm", "layer_norm_backward", "grad_stats", "grad_norm", "grad_clip", "clip_grad_norm",
         "gn_grad_stats", "gn_grad_apply", "gn_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_on_the_current_device_are_taken_others_refused(tbl, name):
    _calls(tbl, 0)[name]()
    assert tbl._lib.calls
    del tbl._lib.calls[:]
    with pytest.raises(ValueError, match="device"):
        _calls(tbl, 1)[name]()
    assert not tbl._lib.calls


MIXED = [("layer_norm", "w"), ("layer_norm", "s"), ("layer_norm_backward", "ws"), ("grad_stats", "recs"),
         ("grad_stats", "grad"), ("grad_norm", "recs"), ("grad_norm", "norm"), ("grad_clip", "recs"),
         ("grad_clip", "norm"), ("grad_clip", "grad"), ("clip_grad_norm", "recs"), ("clip_grad_norm", "norm"),
         ("gn_grad_stats", "grec"), ("gn_grad_apply", "grec"), ("gn_backward", "grec"), ("gn_backward", "part"),
         ("gn_backward", "c")]


@pytest.mark.parametrize("name,other", MIXED)
def test_one_tensor_on_another_device_is_refused(tbl, name, other):
    with pytest.raises(ValueError):
        _calls(tbl, 0, **{other: 1})[name]()
    assert not [c for c in tbl._lib.calls if c != "tb_grad_stats" or other in ("recs", "grad")]


def test_gradients_and_outputs_that_overlap_are_refused(tbl):
    # elements that one CTA writes and another reads or writes would be scaled once or twice, by chance
    buf, a, b, e = t(0, 64), t(0, 8), t(0, 9), t(0, 0)
    for grads, outs in (([a, b, e, e], None),                                # in place; empty ones anywhere
                        (list(buf.split([5, 3, 56])), None),                 # neighbours
                        ([a, a], [buf[:8], buf[8:16]]),                      # one gradient to two places
                        ([buf[:8], buf[8:16]], [buf[:8], buf[16:24]])):      # some in place
        tbl.GradTable(grads, outs)
    for grads, outs in (([a, b, a], None),                                   # a shared parameter's gradient, twice
                        ([buf[:8], buf[7:16]], None),
                        ([a, b[:8]], [buf[:8], buf[:8]]),
                        ([a, b[:8]], [buf[:8], buf[4:12]]),
                        ([buf[:8]], [buf[1:9]]),                             # shifted onto itself
                        ([buf[:8], a], [b[:8], buf[:8]]),                    # onto another's gradient
                        ([buf[:32], a], [buf[32:], buf[8:16]])):
        with pytest.raises(ValueError, match="overlap"):
            tbl.GradTable(grads, outs)

"""The training calls take tensors on the current GPU only: any other is refused by name before
its address reaches a kernel."""
import pytest
import torch

from dspark_block_drafter_gb300 import torch_io as tio

T, H, V, R = 4, 64, 128, 8


def _calls(device):
    """(name of each tensor, a function that makes the call with one of them moved)."""
    dt = dict(device=device)
    f, i = dict(dtype=torch.float32, **dt), dict(dtype=torch.int32, **dt)
    loss = dict(lm_head=torch.ones(V, H, **f), lm_bias=torch.zeros(V, **f),
                d2t=torch.arange(V, **i), markov_w1=torch.ones(V, R, **f),
                markov_w2=torch.ones(R, V, **f), loss=torch.ones(T, **f), total=torch.ones(1, **f),
                n_rows=torch.ones(1, **i), d_hidden=torch.ones(T, H, **f),
                d_lm_head=torch.ones(V, H, **f), d_markov_w1=torch.ones(V, R, **f),
                d_markov_w2=torch.ones(R, V, **f), hidden=torch.ones(T, H, **f),
                prev=torch.zeros(T, **i), labels=torch.zeros(T, **i), weights=torch.ones(T, **f),
                workspace=torch.zeros(1 << 24, dtype=torch.uint8, **dt))

    def head_loss(t):
        head = tio.Head(t["lm_head"], t["markov_w1"], t["markov_w2"], t["lm_bias"], t["d2t"])
        out = tio.LossOutputs(t["loss"], t["total"], t["n_rows"], t["d_hidden"], t["d_lm_head"],
                              t["d_markov_w1"], t["d_markov_w2"])
        tio.head_loss(tio.make_loss_config(T, H, V, R, "f32"), head, t["hidden"], t["prev"],
                      t["labels"], out, t["workspace"], weights=t["weights"])

    rows = ("x", "y", "gate", "x_out", "h", "d_h", "d_x_out", "d_x", "d_y", "d_gate")
    norm = {n: torch.ones(T, H, **f) for n in rows}
    norm.update({n: torch.ones(H, **f) for n in ("w_post", "w_pre", "d_w_post", "d_w_pre")})
    ncfg = tio.make_norm_config(T, H, "f32")

    def block_norm(t):
        tio.block_norm(ncfg, t["x"], t["y"], t["w_pre"], t["h"], t["x_out"], t["gate"], t["w_post"])

    back = dict(norm, workspace=torch.zeros(1 << 24, dtype=torch.uint8, **dt))
    del back["x_out"], back["h"]

    def block_norm_backward(t):
        out = tio.NormGrads(t["d_x"], t["d_y"], t["d_gate"], t["d_w_post"], t["d_w_pre"])
        tio.block_norm_backward(ncfg, t["x"], t["y"], t["w_pre"], t["d_h"], out, t["workspace"],
                                t["d_x_out"], t["gate"], t["w_post"])

    clip = {"gradient 0": torch.ones(9, **f), "outs[0]": torch.ones(9, **f),
            "norm": torch.ones(1, **f), "workspace": torch.zeros(1 << 20, dtype=torch.uint8, **dt)}

    def clip_grads(t):
        gl = tio.GradList([t["gradient 0"]], [t["outs[0]"]])
        tio.clip_grads(gl, 1.0, t["norm"], t["workspace"])

    fore = {n: norm[n] for n in ("x", "y", "gate", "w_post", "w_pre", "x_out", "h")}
    return [(loss, head_loss), (fore, block_norm), (back, block_norm_backward), (clip, clip_grads)]


@pytest.mark.parametrize("which", range(4))
def test_tensors_in_host_memory_are_refused(which):
    tensors, call = _calls("cpu")[which]
    with pytest.raises(ValueError, match="current GPU, got one on cpu"):
        call(tensors)


@pytest.mark.gpu
@pytest.mark.parametrize("which", range(4))
def test_one_tensor_in_host_memory_is_refused_by_name(which):
    tensors, call = _calls("cuda")[which]
    call(tensors)                              # (all on the GPU)
    for name, t in tensors.items():
        with pytest.raises(ValueError, match="(?s)^" + name.replace("[", r"\[") + ": .*got one on cpu"):
            call(dict(tensors, **{name: t.cpu()}))
        with pytest.raises(ValueError, match="(?s)^" + name.replace("[", r"\[") + ": .*got one on cpu"):
            call(dict(tensors, **{name: t.cpu().pin_memory()}))
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("which", [0, 2, 3])
def test_a_workspace_with_gaps_is_refused(which):
    tensors, call = _calls("cuda")[which]
    with pytest.raises(ValueError, match="workspace: need a contiguous"):
        call(dict(tensors, workspace=tensors["workspace"].repeat(2)[::2]))

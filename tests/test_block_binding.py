"""The binding of the attention block's operators refuses host tensors, which a
kernel must never see, in every place a tensor can be given; no GPU is needed:
host tensors that claim a device stand for the ones that are not at fault."""

import pytest
import torch

import rotated_codebook_bit_amd as cq

try:
    cq.lib()
except ImportError:
    pytest.skip("libcq.so is not built", allow_module_level=True)


class OnDevice(torch.Tensor):
    """A host tensor that says it is on device 0, so that the checks of the
    others are reached; a call that passed them all would end in the library's
    own error, not on a GPU (there is none), as its address is misaligned."""

    @staticmethod
    def __new__(cls, t):
        return torch.Tensor._make_subclass(cls, t)

    def get_device(self):
        return 0

    def data_ptr(self):
        return 8


def tensors():
    heads = {name: torch.zeros(4, h, 64) for name, h in (("q", 2), ("k", 1), ("v", 1), ("q_out", 2), ("k_out", 1), ("v_out", 1))}
    return heads, torch.arange(4), torch.ones(32)


CALLS = {
    "rotate": (lambda t: cq.qk_norm_rope(t["q"], t["k"], t["positions"], t["freqs"], t["qw"], t["kw"], v=t["v"], slots=t["slots"], q_out=t["q_out"],
                                         k_out=t["k_out"], v_out=t["v_out"]),
               dict(q=(4, 2, 64), k=(4, 1, 64), v=(4, 1, 64), positions=4, freqs=(32,), qw=(64,), kw=(64,), slots=4, q_out=(4, 2, 64),
                    k_out=(9, 1, 64), v_out=(9, 1, 64))),
    "rotate_grad": (lambda t: cq.qk_norm_rope_grad(t["a"], t["b"], t["q"], t["k"], t["positions"], t["freqs"], t["qw"], t["kw"], dq=t["dq"],
                                                   dk=t["dk"], workspace=t["ws"]),
                    dict(a=(4, 2, 64), b=(4, 1, 64), q=(4, 2, 64), k=(4, 1, 64), positions=4, freqs=(32,), qw=(64,), kw=(64,), dq=(4, 2, 64),
                         dk=(4, 1, 64), ws=(4096,))),
    "attention": (lambda t: cq.attention(t["q"], t["k"], t["v"], q_starts=t["qs"], k_starts=t["ks"], k_lens=t["kl"], out=t["out"], lse=t["lse"],
                                         workspace=t["ws"]),
                  dict(q=(4, 2, 64), k=(9, 1, 64), v=(9, 1, 64), qs=3, ks=2, kl=2, out=(4, 2, 64), lse=(4, 2), ws=(4096,))),
    "attention_alone": (lambda t: cq.attention(t["q"], t["k"], t["v"]), dict(q=(4, 2, 64), k=(9, 1, 64), v=(9, 1, 64))),
    "rotate_alone": (lambda t: cq.qk_norm_rope(t["q"], t["k"], v=t["v"]), dict(q=(4, 2, 64), k=(4, 1, 64), v=(4, 1, 64))),
    "rotate_grad_alone": (lambda t: cq.qk_norm_rope_grad(t["a"], t["b"], t["q"], t["k"]),
                          dict(a=(4, 2, 64), b=(4, 1, 64), q=(4, 2, 64), k=(4, 1, 64))),
    "attention_grad": (lambda t: cq.attention_grad(t["dout"], t["q"], t["k"], t["v"], t["out"], t["lse"], q_starts=t["qs"], k_starts=t["ks"],
                                                   dq=t["dq"], dk=t["dk"], dv=t["dv"], workspace=t["ws"]),
                       dict(dout=(4, 2, 64), q=(4, 2, 64), k=(9, 1, 64), v=(9, 1, 64), out=(4, 2, 64), lse=(4, 2), qs=3, ks=3, dq=(4, 2, 64),
                            dk=(9, 1, 64), dv=(9, 1, 64), ws=(4096,))),
    "logprobs": (lambda t: cq.token_logprobs(t["logits"], t["tokens"]), dict(logits=(4, 50), tokens=4)),
    "logprobs_grad": (lambda t: cq.token_logprobs_grad(t["logits"], t["tokens"], t["lse"], t["g"], t["h"], t["entropy"], dlogits=t["out"]),
                      dict(logits=(4, 50), tokens=4, lse=(4,), g=(4,), h=(4,), entropy=(4,), out=(4, 50))),
}


def make(shape):
    return torch.zeros(shape, dtype=torch.int64) if isinstance(shape, int) else torch.zeros(shape)


@pytest.mark.parametrize("name", CALLS)
def test_a_host_tensor_in_any_place(name):
    call, shapes = CALLS[name]
    for at_fault in shapes:
        t = {key: make(shape) if key == at_fault else OnDevice(make(shape)) for key, shape in shapes.items()}
        with pytest.raises(ValueError, match="CUDA|device"):
            call(t)
    with pytest.raises(ValueError):
        call({key: make(shape) for key, shape in shapes.items()})

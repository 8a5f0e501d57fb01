"""Refusals of the queries' and keys' norm and rotation, on the CPU: nothing is enqueued."""
import os

import pytest
import torch

import precision_block_scaled_amd as P
from precision_block_scaled_amd import pipeline as PL

pytestmark = pytest.mark.skipif(not os.path.exists(P.lib_path), reason="libpbs.so is not built")

BF, F32 = P.PBS_FMT_BF16, P.PBS_FMT_F32
A = 1 << 20                     # addresses that no call reads
GOOD = dict(q=A, q_strides=(5120, 640, 128), heads=4, k=2 * A, k_strides=(5120, 640, 128), kv_heads=1, x_fmt=BF, batch=2,
            seq=8, head_dim=128, q_weight=3 * A, k_weight=4 * A, w_fmt=BF, norm=1, eps=1e-6, positions=5 * A,
            pos_batch_stride=8, freqs=6 * A, rot_dim=128, interleaved=0, q_out=7 * A, q_out_strides=(4096, 512, 128),
            k_out=8 * A, k_out_strides=(1024, 128, 128), y_fmt=BF, stream=0)
BAD = [
    (dict(x_fmt=P.PBS_FMT_E4M3), 3, "formats"), (dict(y_fmt=P.PBS_FMT_E2M1), 3, "formats"), (dict(w_fmt=9), 3, "formats"),
    (dict(head_dim=0), 2, "head_dim"), (dict(head_dim=513), 2, "head_dim"), (dict(batch=-1), 2, "batch"),
    (dict(seq=-1), 2, "batch"), (dict(heads=-1), 2, "heads"), (dict(kv_heads=70000), 2, "heads"),
    (dict(batch=1 << 20, seq=1 << 20), 2, "2^30"), (dict(rot_dim=130), 2, "rot_dim"), (dict(rot_dim=7), 2, "rot_dim"),
    (dict(rot_dim=-2), 2, "rot_dim"), (dict(freqs=None), 1, "freqs"), (dict(freqs=6 * A + 4), 1, "freqs"),
    (dict(positions=5 * A + 4), 1, "positions"), (dict(pos_batch_stride=7), 2, "positions"),
    (dict(pos_batch_stride=-8), 2, "positions"), (dict(eps=-1.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"),
    (dict(eps=float("inf")), 1, "eps"), (dict(q=None), 1, "q is null"), (dict(k_out=None), 1, "k_out is null"),
    (dict(q=A + 1), 1, "aligned"), (dict(q_weight=3 * A + 1), 1, "aligned"), (dict(q_strides=None), 1, "strides"),
    (dict(k_out_strides=None), 1, "strides"), (dict(q_strides=(5120, -640, 128)), 2, "strides"),
    (dict(q_out_strides=(4096, 512, 127)), 2, "overlap"), (dict(q_out_strides=(4096, 0, 128)), 2, "overlap"),
    (dict(q_out_strides=(4095, 512, 128)), 2, "overlap"), (dict(k_out_strides=(0, 128, 128)), 2, "overlap"),
    (dict(q_out=A), 1, "input's memory"), (dict(k_out=A), 1, "input's memory"),
    (dict(q_out=A, q_out_strides=(5120, 640, 128), y_fmt=F32), 1, "input's memory"),
]


@pytest.mark.parametrize("change,status,text", BAD, ids=lambda v: str(v)[:40])
def test_forward_refusals(change, status, text):
    with pytest.raises(P.PBSError, match=text.replace("^", r"\^")) as e:
        P.pbs_qk_norm_rope(**{**GOOD, **change})
    assert e.value.status == status


GRAD = dict(dq=9 * A, dq_strides=(4096, 512, 128), dk=10 * A, dk_strides=(1024, 128, 128), dv=11 * A,
            dv_strides=(1024, 128, 128), y_fmt=BF, **{k: v for k, v in GOOD.items() if k in (
                "q", "q_strides", "heads", "k", "k_strides", "kv_heads", "x_fmt", "batch", "seq", "head_dim", "q_weight",
                "k_weight", "w_fmt", "norm", "eps", "positions", "pos_batch_stride", "freqs", "rot_dim", "interleaved")},
            dq_out=12 * A, dq_out_strides=(6144, 768, 128), dk_out=12 * A + 1024, dk_out_strides=(6144, 768, 128),
            dv_out=12 * A + 1280, dv_out_strides=(6144, 768, 128), dq_weight=13 * A, dk_weight=14 * A, amax_out=15 * A,
            workspace=16 * A, workspace_bytes=1 << 20, stream=0)
GRAD_BAD = [
    (dict(y_fmt=P.PBS_FMT_E5M2), 3, "formats"), (dict(dq=None), 1, "dq is null"), (dict(dk_out=None), 1, "dk_out is null"),
    (dict(dv=None), 1, "go together"), (dict(dv_out=None), 1, "go together"), (dict(dv_strides=None), 1, "strides"),
    (dict(dq_weight=13 * A + 2), 1, "aligned"), (dict(amax_out=15 * A + 1), 1, "aligned"),
    (dict(workspace=None), 1, "workspace"), (dict(workspace=16 * A + 8), 1, "workspace"), (dict(workspace_bytes=64), 1, "workspace"),
    (dict(dq_out=A), 1, "input's memory"), (dict(dq_out=9 * A), 1, "input's memory"), (dict(dv_out=9 * A), 1, "input's memory"),
    (dict(dv_out=2 * A), 1, "input's memory"), (dict(dq_out_strides=(6144, 768, 64)), 2, "overlap"),
    (dict(rot_dim=200), 2, "rot_dim"),
]


@pytest.mark.parametrize("change,status,text", GRAD_BAD, ids=lambda v: str(v)[:40])
def test_gradient_refusals(change, status, text):
    with pytest.raises(P.PBSError, match=text) as e:
        P.pbs_qk_norm_rope_grad(**{**GRAD, **change})
    assert e.value.status == status


def test_workspace_bytes():
    assert P.pbs_qk_norm_rope_grad_bytes(0, 5, 128) == (2 * 128 + 3) * 4
    assert P.pbs_qk_norm_rope_grad_bytes(31, 512, 128) == 768 * (2 * 128 + 3) * 4
    for bad in ((-1, 1, 128), (1, 1, 0), (1, 1, 513), (1 << 24, 1 << 24, 64)):
        with pytest.raises(P.PBSError):
            P.pbs_qk_norm_rope_grad_bytes(*bad)


def test_python_refusals():
    q, k = torch.zeros(2, 8, 4, 16), torch.zeros(2, 8, 2, 16)
    w, f = torch.ones(16), PL.rope_frequencies(16, device="cpu")
    pos = torch.zeros(2, 8, dtype=torch.int64)
    bad = [dict(q=q[0]), dict(q=q.half()), dict(q=q.transpose(2, 3)), dict(k=k[:, :7]), dict(k=k.bfloat16()), dict(k=k[0]),
           dict(q_weight=w[:8]), dict(q_weight=w.double()), dict(q_weight=w.bfloat16()), dict(k_weight=w, k=None),
           dict(positions=pos.int()), dict(positions=pos[:1, :7]), dict(positions=pos.t()), dict(freqs=f.float()),
           dict(positions=torch.zeros(8, 2, dtype=torch.int64).t()), dict(freqs=torch.cat((f, f))), dict(freqs=f[None]),
           dict(out_dtype=torch.float16), dict(q_out=q[:1]), dict(k_out=k[:, :, :1]), dict(k=None, k_out=k),
           dict(q_out=q.bfloat16(), k_out=k), dict(q=None)]
    for change in bad:
        with pytest.raises(ValueError):
            PL.qk_norm_rope(**{**dict(q=q, k=k, q_weight=w, k_weight=w, positions=pos, freqs=f), **change})
    good = dict(dq=q, dk=k, q=q, k=k, q_weight=w, k_weight=w, positions=pos, freqs=f)
    for change in (dict(dq=None), dict(dk=None), dict(k=None), dict(dv=k), dict(dv_out=k), dict(dq=q[:1]),
                   dict(dk=k.bfloat16()), dict(dq_out=q.bfloat16()), dict(dv=k, dv_out=k.bfloat16()),
                   dict(amax=torch.zeros(2)), dict(dk_out=k[:, :, :1])):
        with pytest.raises(ValueError):
            PL.qk_norm_rope_grad(**{**good, **change})
    with pytest.raises(ValueError, match="on the GPU"):
        PL.qk_norm_rope(q, k, w, w, pos, f)
    with pytest.raises(ValueError, match="on the GPU"):
        PL.qk_norm_rope_grad(**good)
    with pytest.raises(ValueError):
        PL.rope_frequencies(7)
    assert PL.rope_frequencies(4, 100.0, "cpu").tolist() == [1.0, 100.0 ** -0.5]


def test_outputs_on_one_tensor():
    with pytest.raises(P.PBSError, match="q_out and k_out are one tensor") as e:
        P.pbs_qk_norm_rope(**{**GOOD, "k_out": GOOD["q_out"]})
    assert e.value.status == 1
    for change, text in ((dict(dk_out=12 * A), "dq_out and dk_out"), (dict(dv_out=12 * A), "dv_out and dq_out"),
                         (dict(dv_out=12 * A + 1024), "dk_out and dv_out"), (dict(dk_weight=13 * A), "dq_weight and dk_weight")):
        with pytest.raises(P.PBSError, match=text + " are one") as e:
            P.pbs_qk_norm_rope_grad(**{**GRAD, **change})
        assert e.value.status == 1

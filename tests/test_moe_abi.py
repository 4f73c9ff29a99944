"""The mixture-of-experts entry points on the CPU: declarations, and every
argument outside the contract refused before any device is touched."""
import ctypes
import os
import re

import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
from dense_tiled_gemm_fp16_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = [0x7F0000000000 + (i << 36) for i in range(8)]   # never dereferenced


def test_header_declares_the_binding_list():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gemm_moe.h")).read(), flags=re.S)
    assert sorted(set(re.findall(r"^\s*\w+\s+(gemm_\w+)\s*\(", text, re.M))) == sorted(_lib.EXPORTS_MOE)
    fields = re.findall(r"(\w+)\s*[,;]", text[text.index("typedef struct"):text.index("} gemm_moe_args")])
    assert fields == [f for f, _ in _lib.MoeArgs._fields_]
    for name, value in (("TOKENS", g.moe.MAX_TOKENS), ("EXPERTS", g.moe.MAX_EXPERTS), ("TOP_K", g.moe.MAX_TOP_K)):
        assert re.search(rf"GEMM_MOE_MAX_{name} {value}\b", text)


def call(ws=P[7], nws=1 << 30, **kw):
    a = dict(X=P[0], ldx=70, logits=P[1], ldl=6, W1=P[2], w1_e=80 * 70, w1_n=70, S1=None, s1_e=0, s1_n=0,
             W2=P[3], w2_e=70 * 40, w2_n=40, S2=None, s2_e=0, s2_n=0, Y=P[4], ldy=70, T=5, E=6, H=70, I=40,
             top_k=2, fmt=1, fmt_logits=2, mx4=0, renormalize=1)
    a.update(kw)
    return g.lib.gemm_moe(ctypes.byref(_lib.MoeArgs(**a)), None, ws, nws)


MX = dict(mx4=1, w1_e=80 * 48, w1_n=48, S1=P[5], s1_e=80 * 3, s1_n=3, w2_e=70 * 32, w2_n=32, S2=P[6],
          s2_e=70 * 2, s2_n=2)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), -1), (dict(logits=None), -1), (dict(W1=None), -1), (dict(W2=None), -1), (dict(Y=None), -1),
    ({**MX, "S1": None}, -1), ({**MX, "S2": None}, -1),
    (dict(T=0), -2), (dict(T=65), -2), (dict(E=0), -2), (dict(E=513), -2), (dict(top_k=0), -2),
    (dict(top_k=7), -2), (dict(E=40, ldl=40, top_k=17), -2), (dict(H=0), -2), (dict(I=-1), -2),
    (dict(H=2 ** 31), -2), (dict(H=2 ** 26 + 1, ldx=2 ** 27, w1_n=2 ** 20, w1_e=2 ** 27, w2_e=2 ** 33, ldy=2 ** 27), -2), (dict(w1_e=2 ** 61), -2), (dict(w2_n=2 ** 57), -2),
    (dict(fmt=2), -7), (dict(fmt_logits=3), -7), (dict(mx4=2), -7),
    (dict(ldx=0), -3), (dict(ldl=-1), -3), (dict(w1_n=0), -3), (dict(w2_e=-1), -3),
    ({**MX, "w1_n": 47}, -3), ({**MX, "s1_n": 2}, -3), ({**MX, "w2_n": 16}, -3), ({**MX, "s2_n": 1}, -3),
    (dict(ldy=69), -4),
    (dict(Y=P[0] + 2), -5), (dict(Y=P[1]), -5), (dict(Y=P[2] + 64), -5), (dict(Y=P[3]), -5),
    ({**MX, "Y": P[5] + 8}, -5), ({**MX, "Y": P[6]}, -5), (dict(ws=P[4]), -5), (dict(ws=P[3]), -5),
    (dict(ldx=2 ** 30), -9), (dict(w1_n=2 ** 26, w1_e=2 ** 33), -9), (dict(w2_n=2 ** 27, w2_e=2 ** 35), -9),
    ({**MX, "s1_n": 2 ** 27}, -9), ({**MX, "s2_n": 2 ** 28}, -9), (dict(I=2 ** 20 + 1), -2),
    (dict(nws=100), -6), (dict(ws=P[7] + 16), -6),
])
def test_refusals(kw, code):
    assert call(**kw) == code


def test_null_args():
    assert g.lib.gemm_moe(None, None, None, 0) == -1


def test_workspace_bytes():
    assert g.gemm_moe_workspace_bytes(0, 4, 2, 64, 64) == 0
    assert g.gemm_moe_workspace_bytes(65, 4, 2, 64, 64) == 0
    assert g.gemm_moe_workspace_bytes(4, 4, 5, 64, 64) == 0
    n = g.gemm_moe_workspace_bytes(4, 8, 2, 100, 33)
    assert n >= 2 * 8 * 40 * 2 + 8 * 8 and n % 256 == 0


def test_python_refusals():
    x, logits = torch.zeros(2, 32, dtype=torch.float16), torch.zeros(2, 4)
    up, down = torch.zeros(4, 64, 32, dtype=torch.float16), torch.zeros(4, 32, 32, dtype=torch.float16)
    with pytest.raises(ValueError):
        g.gemm_moe(x, logits, up, down, 2)           # not on a GPU
    with pytest.raises(TypeError):
        g.gemm_moe(x, logits, up.bfloat16(), down, 2)
    with pytest.raises(TypeError):
        g.gemm_moe(x.float(), logits, up, down, 2)
    with pytest.raises(ValueError):
        g.gemm_moe(x[0], logits, up, down, 2)
    q = g.MX4(torch.zeros(4, 64, 16, dtype=torch.uint8), torch.zeros(4, 64, 1, dtype=torch.uint8), 32)
    with pytest.raises(TypeError):
        g.gemm_moe(x, logits, q, down, 2)

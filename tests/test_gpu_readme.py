"""The README's serving example runs as it is printed, and gives what the calls' oracle-tested parts give."""
import os
import re

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def _block(after):
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        text = f.read()
    return re.search(r"```python\n(.*?)```", text[text.index(after):], re.S).group(1)


@pytest.mark.parametrize("columns", [False, True])
def test_the_serving_example(lib, columns):
    B, Hq, Hkv, d, T = 2, 8, 2, 128, 90
    n = [70, T]
    N = sum(n)
    rows = torch.randn(N, Hq + 2 * Hkv, d, device="cuda").to(torch.bfloat16)
    q, k, v = rows.split([Hq, Hkv, Hkv], 1) if columns else (x.contiguous() for x in rows.split([Hq, Hkv, Hkv], 1))
    need = -(-max(n) // 32)
    cu = torch.tensor(np.cumsum([0] + n), **I32)
    names = dict(
        torch=torch, cpa=lib, q=q, k=k, v=v, cu=cu, start=torch.zeros(B, **I32), zeros=torch.zeros(B, **I32), cu_kv=cu, Nkv=N,
        k4=torch.zeros(2, B * need, Hkv, 9 * d, dtype=torch.uint8, device="cuda"),
        v4=torch.zeros(2, B * need, Hkv, 9 * d, dtype=torch.uint8, device="cuda"),
        bt=torch.arange(B * need, **I32).reshape(1, B, need).repeat(2, 1, 1), f=10000.0 ** (-torch.arange(64, device="cuda").double() / 64),
        T=T, B=B, Hq=Hq, Hkv=Hkv, d=d, max_len=max(n), sl=torch.tensor(n, **I32))
    code = _block("Serving a model with rotary positions").split("# decode:")
    exec(code[0], names)
    whole = names["q"]
    names["q"] = whole[cu[1:].long() - 1].contiguous()   # the last tokens' queries, as a decode step has them
    prefill = names["out"][cu[1:].long() - 1]
    exec("#" + code[1], names)
    # both attend the same 4-bit context; the read-back rounds K and V to bf16 once more: 2^-9 of a score's |q||k|
    # (a few units) and of V, and the weights 2^-9: far below 1/16 of the largest value
    assert bool(torch.isfinite(names["out"].float()).all())
    assert float((names["out"].float() - prefill.float()).abs().max()) <= 2.0 ** -4 * float(v.float().abs().max())

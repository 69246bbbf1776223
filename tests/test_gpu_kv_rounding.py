"""Scales that are no power of two, where a quotient rounded to binary32 first would meet a tie of e4m3's."""
import numpy as np
import pytest
import torch

from kv_ref import F8
from test_gpu_kv import _built, check_append, cuda_int, fresh, ok  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def near_ties(quotient):
    """(x in bf16's significands, binary32 s) with x / s, or x * s, beside a tie of e4m3's on either side of it, but on it
    once rounded to binary32."""
    found = []
    for t in range(17, 32, 2):                                   # ties: odd multiples of 1/16 in [1, 2)
        for m in range(128, 256) if quotient else range(8, 16):
            x = m / (128 if quotient else 8)
            s = np.float32(x / (t / 16) if quotient else t / 16 / x)
            exact = x / float(s) if quotient else x * float(s)
            binary32 = np.float32(x) / s if quotient else np.float32(x) * s
            if binary32 == t / 16 and exact != t / 16:
                found.append((x, float(s), t, exact > t / 16))
    return found


def test_stored_values_round_once():
    """x / scale, the scale the caller's: towards the side of the tie that it is on."""
    cases = near_ties(True)
    assert {(t, up) for _, _, t, up in cases} >= {(17, True), (19, False)}
    cpu, dev, kv = fresh(R=1, H=1, D=64, P=16, pages=len(cases), q_heads=1)
    slots, x = [], torch.zeros(1, len(cases), 1, 64)
    for i, (v, s, _, _) in enumerate(cases):
        for scale in (cpu[2], cpu[3], dev[2], dev[3]):
            scale[0, i] = s
        x[0, i, 0] = v * torch.tensor([1.0, -1.0] * 32) * 2.0 ** (torch.arange(64) // 2 % 12 - 6)
        slots.append(16 * i + 3)
    x = x.to(torch.bfloat16)
    kv.append(x.cuda(), x.cuda(), cuda_int(slots))
    ok(kv)
    check_append(cpu, dev, [x, x], slots)


def test_held_values_round_once():
    """value * (old scale / new scale) when a page's scale grows."""
    cases = near_ties(False)
    assert any(up for *_, up in cases) and any(not up for *_, up in cases)
    cpu, dev, kv = fresh(R=1, H=1, D=64, P=16, pages=len(cases), q_heads=1)
    slots, x = [], torch.full((1, len(cases), 1, 64), 448.0 * 4, dtype=torch.bfloat16)          # grows the scale to 4
    for i, (v, s, _, _) in enumerate(cases):
        for scale in (cpu[2], cpu[3], dev[2], dev[3]):
            scale[0, i] = s
        held = (v * torch.tensor([1.0, -1.0] * 32) * 2.0 ** (torch.arange(64) // 2 % 7)).to(F8)
        for c in (cpu[0], cpu[1], dev[0], dev[1]):
            c[0, i, 0, :5] = held.to(c.device)
        slots.append(16 * i + 5)
    kv.append(x.cuda(), x.cuda(), cuda_int(slots))
    ok(kv)
    check_append(cpu, dev, [x, x], slots)

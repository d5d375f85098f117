"""The give-up path of the paged tree attention's bounded waits, made to run on
purpose: with the first-wait limit lowered to a few clock cycles the waits for
tiles and products run out.  What a CTA could not finish is NaN, everything else
is as it was, medusa_device_status reports it once, and with the default limit the
next calls give the same bits as before."""
import numpy as np
import pytest
import torch

from test_parity_q8 import NAMES, attention_case, dev
from util import to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,N,Hq,Hkv,D,P,lens", [
    (2, 1, 8, 2, 128, 64, [900, 30]),         # blocks of 16 rows
    (3, 40, 4, 4, 64, 16, [2000, 0, 333]),    # of 64
    (2, 150, 4, 4, 128, 32, [1500, 77]),      # of 128, the streams share tiles
    (2, 20, 4, 2, 128, 64, [100, 30]),        # units that are not cut
])
def test_wait_give_up_is_reported_and_the_next_calls_are_correct(medusa, B, N, Hq, Hkv, D, P, lens):
    M = medusa
    c = attention_case(41, B, N, Hq, Hkv, D, P, lens, "bf16")
    t = [dev(c[n], "bf16") for n in ("q", "k_tree", "v_tree")] + [to_dev(c[n]) for n in NAMES + ("table", "kv_len", "mask")]

    def run():
        out = M.tree_attention_q8(*t, c["scale"])
        torch.cuda.synchronize()
        return out.float().cpu().numpy()

    M.device_status()  # clear whatever an earlier test left
    before = run()
    M.device_status()
    assert np.isfinite(before).all()
    try:
        M.set_wait_limit(4)
        hurt = run()
    finally:
        M.set_wait_limit(0)
    with pytest.raises(M.MedusaError) as e:
        M.device_status()
    assert e.value.code == -5
    assert np.isnan(hurt).any() and (np.isnan(hurt) | (hurt == before)).all()
    assert np.array_equal(run(), before)
    M.device_status()

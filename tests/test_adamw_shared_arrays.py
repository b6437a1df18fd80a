"""AdamW refuses one array in two places of a tensor: no GPU, nothing is enqueued."""
import pytest

from sparse_linear_layers_bitlinear_b200 import build, sbl

A = 0x10000  # aligned addresses that nothing reads
DISTINCT = dict(w=A, master=A + 0x1000, grad=A + 0x2000, m=A + 0x3000, v=A + 0x4000, m_scale=A + 0x5000, v_scale=A + 0x6000)


@pytest.mark.parametrize("same,bits", [(("m", "v"), 32), (("m", "w"), 32), (("v", "w"), 32), (("master", "m"), 32),
                                       (("master", "v"), 32), (("master", "w"), 32), (("grad", "m"), 32),
                                       (("grad", "w"), 32), (("m_scale", "master"), 8), (("m_scale", "v_scale"), 8), (("m", "v"), 8)])
def test_one_array_in_two_places(same, bits):
    build.build()
    arr = (sbl.sbl_adamw_tensor * 1)()
    for name, at in DISTINCT.items():
        setattr(arr[0], name, at)
    setattr(arr[0], same[0], DISTINCT[same[1]])
    arr[0].numel, arr[0].flags = 512, sbl.SBL_ADAMW_STATE_8BIT if bits == 8 else 0
    params = sbl._ADAMW_PARAMS.pack(1e-3, 0.9, 0.95, 1e-8, 0.1, 1, 0, 0, 0)
    assert sbl.lib().sbl_adamw_step(arr, 1, params, None, None) == sbl.SBL_ERR_INVALID_ARG

"""The gated scan's bounded waits: a block that never gets what it waits for gives up, the launch ends,
the device-wide status reports it once, and the next call is right.  No GPU fault is involved: a block
withholds its sums from its cluster, or skips the fetch of its first tile."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

POLLS = 2000  # under a millisecond or so each wait


# full clusters of eight over several strides (tiles by TMA, by copies, and with gy in a ring of its own in
# bf16), clusters that pairs of channels fill, single blocks
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,sums,tiles", [((1, 16384, 64), (0, 3, 7), (0, 2)), ((1, 16384, 33), (1,), (0, 5)), ((1, 300, 64), (1,), (1,)),
                                              ((1, 4100, 4040), (0,), (1,)), ((40, 700, 768), (), (0,)), ((20, 1000, 999), (), (0,))],
                         ids=lambda v: "x".join(map(str, v)) if v else "none")
def test_withheld_data_times_out_and_the_next_call_is_right(shape, sums, tiles, dtype):
    import torch
    import linear_attention_rnn_wkv_b200 as wkv
    L = wkv.lib()
    td, io = (torch.float32, 0) if dtype == "f32" else (torch.bfloat16, 1)
    r = np.random.default_rng(800)
    g, x, gy = (torch.from_numpy(r.normal(1, 1, shape).astype(np.float32)).cuda().to(td) for _ in range(3))

    def normal():
        y, so, carry = wkv.gated_scan_forward(g, x, want_carry=True)
        return (y, so, carry) + wkv.gated_scan_backward(g, x, carry, gy)

    ref = normal()
    stream = torch.cuda.current_stream().cuda_stream
    L.wkv_get_device_status(stream)  # start from a clear word
    out = [torch.empty_like(g) for _ in range(2)]
    for backward in (False, True):
        for drop in [(k, -1) for k in sums] + [(-1, k) for k in tiles]:
            st = L.wkv_testhook_gated_scan_drop(*shape, io, g.data_ptr(), x.data_ptr(), ref[2].data_ptr(),
                                                gy.data_ptr() if backward else None, out[0].data_ptr(),
                                                out[1].data_ptr(), *drop, POLLS, stream)
            assert st == 0
            assert L.wkv_get_device_status(stream) == 5, f"backward {backward}, drop {drop}"  # WKV_ERR_TIMEOUT
            assert L.wkv_get_device_status(stream) == 0
            assert all(torch.equal(a, b) for a, b in zip(normal(), ref)), f"after backward {backward}, drop {drop}"
            assert L.wkv_get_device_status(stream) == 0


def test_nothing_withheld_is_the_normal_call():
    """The hook without a drop: the same bits, no status."""
    import torch
    import linear_attention_rnn_wkv_b200 as wkv
    L = wkv.lib()
    g, x, gy = (torch.randn(1, 5000, 96, device="cuda") for _ in range(3))
    y, _, carry = wkv.gated_scan_forward(g, x, want_carry=True)
    gg, gx, _ = wkv.gated_scan_backward(g, x, carry, gy)
    stream = torch.cuda.current_stream().cuda_stream
    L.wkv_get_device_status(stream)
    a, b, c = (torch.empty_like(g) for _ in range(3))
    for args in ((None, a, None), (gy.data_ptr(), b, c)):
        assert L.wkv_testhook_gated_scan_drop(1, 5000, 96, 0, g.data_ptr(), x.data_ptr(), carry.data_ptr(), args[0], args[1].data_ptr(),
                                              args[2].data_ptr() if args[2] is not None else None, -1, -1, 1 << 18, stream) == 0
    assert L.wkv_get_device_status(stream) == 0
    assert torch.equal(a, y) and torch.equal(b, gx) and torch.equal(c, gg)

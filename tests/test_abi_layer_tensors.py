"""The tensor calls of the 4-bit experts refuse tensors that a kernel would misread, before anything
is launched.  CPU only: the last refusal, of tensors that are otherwise right, is their device."""
import pytest
import torch

from test_abi_host import moe  # noqa: F401  (the built library)

T, H, E, K, I = 6, 256, 8, 2, 384  # (at I = H / 2 the two operands have one size)


def arguments(moe):  # noqa: F811
    d = moe.dims(T, H, E, K, I)
    return dict(x=torch.zeros((T, H), dtype=torch.bfloat16), w_router=torch.zeros((H, E)), bias=torch.zeros(E),
                packed_gate_up=torch.zeros(moe.moe_mx4_packed_bytes(E, H, 2 * I), dtype=torch.uint8),
                packed_down=torch.zeros(moe.moe_mx4_packed_bytes(E, I, H), dtype=torch.uint8), d=d,
                workspace=torch.zeros(moe.moe_mx4_layer_workspace_bytes(d) + 1024, dtype=torch.uint8))


def test_layer_refuses_what_it_would_misread(moe):  # noqa: F811
    good = arguments(moe)

    def refused(match, error=ValueError, **bad):
        with pytest.raises(error, match=match):
            moe.mx4_layer_forward(**{**good, **bad})

    refused("x:", x=good["x"].float())
    refused("x:", x=good["x"][:5])
    refused("x:", x=torch.zeros((T, 2 * H), dtype=torch.bfloat16)[:, ::2])
    refused("w_router:", w_router=good["w_router"].bfloat16())
    refused("w_router:", w_router=torch.zeros((E, H)).t())
    refused("w_router:", w_router=torch.zeros((E, H)))
    refused("bias:", bias=torch.zeros(E - 1))
    refused("bias:", bias=torch.zeros(E, dtype=torch.float64))
    refused("packed_gate_up:", packed_gate_up=good["packed_gate_up"][:-256])
    refused("packed_down:", packed_down=good["packed_gate_up"])
    refused("packed_gate_up:", packed_gate_up=good["packed_down"], packed_down=good["packed_gate_up"])
    refused("packed_down:", packed_down=torch.zeros((good["packed_down"].numel(), 2), dtype=torch.uint8)[:, 0])
    refused("workspace:", workspace=torch.zeros((good["workspace"].numel(), 2), dtype=torch.uint8)[:, 0])
    refused("workspace:", TypeError, workspace=None)
    refused("x:", TypeError, x=None)
    refused("opts", TypeError, opts=moe.router_opts())
    refused("CUDA device")


@pytest.mark.gpu
def test_dims_outside_the_limits_keep_their_status(moe, cuda_ok):  # noqa: F811
    good = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in arguments(moe).items()}
    for d, code in ((moe.dims(T, 200, E, K, I), "UNSUPPORTED"), (moe.dims(T, 256, E, E + 1, I), "INVALID_ARG")):
        with pytest.raises(moe.MoEError) as e:
            moe.mx4_layer_forward(**{**good, "d": d, "w_router": torch.zeros((d.H, E), device="cuda"),
                                     "x": torch.zeros((T, d.H), dtype=torch.bfloat16, device="cuda")})
        assert moe.STATUS[e.value.code] == "MOE_ERR_" + code
    for other in ("x", "bias", "packed_down", "workspace"):
        with pytest.raises(ValueError, match="device"):
            moe.mx4_layer_forward(**{**good, other: good[other].cpu()})


def test_product_refuses_strided_operands(moe):  # noqa: F811
    N = 256
    x, off = torch.zeros((T, H)), torch.zeros(E + 1, dtype=torch.int32)
    n, ws = moe.moe_mx4_packed_bytes(E, H, N), torch.zeros(1 << 20, dtype=torch.uint8)
    packed = torch.zeros(n, dtype=torch.uint8)
    with pytest.raises(ValueError, match="packed:"):
        moe.mx4_expert_product(x, off, torch.zeros((n, 2), dtype=torch.uint8)[:, 0], N, ws)
    with pytest.raises(ValueError, match="workspace:"):
        moe.mx4_expert_product(x, off, packed, N, torch.zeros((1 << 20, 2), dtype=torch.uint8)[:, 0])
    with pytest.raises(TypeError, match="workspace:"):
        moe.mx4_expert_product(x, off, packed, N, None)
    with pytest.raises(ValueError, match="CUDA device"):
        moe.mx4_expert_product(x, off, packed, N, ws)


def test_selection_options_are_the_selections(moe):  # noqa: F811
    """The router's options are another, shorter structure."""
    l = torch.zeros((T, E))
    idx, w = torch.zeros((T, K), dtype=torch.int32), torch.zeros((T, K))
    for bad in (moe.router_opts(), bytes(20), 3):
        with pytest.raises(TypeError, match="opts"):
            moe.route_select(l, K, bad)
        with pytest.raises(TypeError, match="opts"):
            moe.route_select_backward(l, idx, w, bad)
        with pytest.raises(TypeError, match="opts"):
            moe.moe_route_select(4096, 0, E, None, bad, T, E, K, 4096, 4096, stream=0)


@pytest.mark.parametrize("experts,k,code", [
    (E, 1 << 40, "INVALID_ARG"), (E, E + 1, "INVALID_ARG"), (E, 0, "INVALID_ARG"), (E, -1, "INVALID_ARG"),
    (64, 17, "UNSUPPORTED"), (300, 4, "UNSUPPORTED")])
def test_a_choice_outside_the_limits_is_refused_before_it_is_allocated(moe, experts, k, code):  # noqa: F811
    with pytest.raises(moe.MoEError) as e:
        moe.route_select(torch.zeros((T, experts)), k)
    assert moe.STATUS[e.value.code] == "MOE_ERR_" + code


@pytest.mark.gpu
@pytest.mark.parametrize("k", [1 << 40, 1 << 30, 17, 0, -1])
def test_a_choice_outside_the_limits_on_both_paths(moe, cuda_ok, k):  # noqa: F811
    wide = torch.zeros((4096, 72), device="cuda")
    torch.cuda.reset_peak_memory_stats()
    for l in (wide[:, :64], wide[:, :64].contiguous()):
        held = torch.cuda.max_memory_allocated()
        with pytest.raises(moe.MoEError):
            moe.route_select(l, k)
        assert torch.cuda.max_memory_allocated() == held

"""A cache of one scale whose products with the codes do not fit bf16, so that rows
that are exact differ from rows that are rounded."""
import torch

ODD = 0.0213   # (codes have four significant bits: a scale of up to four more would fit bf16's eight)


def odd_scale(c, scale=ODD):
    """The given tests' Cache ("fp8_tensor") with another scale."""
    c.scales = torch.tensor([scale])
    codes = c.data.view(torch.float8_e4m3fn)
    c.exact = codes.double() * c.scales.double()
    c.seen = (codes.float() * c.scales).to(torch.bfloat16).double()
    return c

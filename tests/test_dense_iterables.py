"""An update set takes its tensors from any iterable, as from lists (CPU checks)."""
import torch

import mxfp4_precision_numerics_amd as mxq
from test_dense_checks import lists, stub  # noqa: F401


def test_an_update_set_takes_iterators(stub):  # noqa: F811
    for eight in (False, True):
        a = lists(eight=eight)
        s = mxq.AdamW(**{name: iter(ts) for name, ts in a.items()}, decay=iter([True, False]))
        listed = mxq.AdamW(**a, decay=[True, False])
        assert s.chunks == listed.chunks and all(x is y for x, y in zip(s.params, a["params"]))
        n = 11 * len(a["params"])  # a tensor's words in the table
        assert torch.equal(torch.Tensor(s._tables)[:n], torch.Tensor(listed._tables)[:n])


def test_an_update_set_takes_a_modules_parameters(stub):  # noqa: F811
    """parameters() is a generator."""
    a = lists(eight=False)
    module = type("Module", (), {"parameters": lambda self: (p for p in a["params"])})()
    rest = {name: ts for name, ts in a.items() if name != "params"}
    assert mxq.AdamW(module.parameters(), **rest).params == a["params"]
    assert mxq.GradientSet(p for p in a["grads"]).grads == a["grads"]

"""Name of the Python module that ``csrc/binding.cpp`` is built into."""
import re

import torch


def native_name() -> str:
    """For this torch: its version and the commit that it was built of."""
    commit = str(getattr(torch.version, "git_version", None))[:12]
    return "_native_torch_" + re.sub(r"\W", "_", f"{torch.__version__}_{commit}")
